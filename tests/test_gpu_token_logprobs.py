"""token_logprobs and token_logprobs_backward against the definitions in 64 bits,
at the sizes, layouts and masks where they can go wrong.

Tolerances. A lane adds up to V / 256 terms one after another and the lanes join in
12 more sums, so the sum of exponentials is within (V / 256 + 64) 2^-23 of its value;
the distance to the maximum carries two roundings, at most 2^-22 of itself. The
gradient's probabilities inherit the rounding of logsumexp (|logsumexp| 2^-24 in the
exponent) beside a few of their own, and a bfloat16 result one more of 2^-9.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

import sparse_embedding_weight_amd as ewg  # noqa: E402

NEG = -math.inf


@pytest.fixture(autouse=True)
def _gpu(require_gpu):
    yield


def reference(logits, targets, top_k, temperature):
    """The definitions in 64 bits on the CPU; masks as documented."""
    x = logits.detach().cpu().double()
    t = targets.cpu().long()
    bad = torch.isnan(x).any(1) | (x == math.inf).any(1)
    y = torch.where(x <= -1e38, torch.full_like(x, NEG), x) / temperature
    m = y.amax(1)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(y - m0[:, None])
    s = e.sum(1)
    lse = m0 + torch.log(s)
    empty = s == 0
    p = torch.where(empty[:, None], torch.zeros_like(e), e / s.clamp(min=1e-300)[:, None])
    entropy = -torch.xlogy(p, p).sum(1)
    lp = y.gather(1, t.clamp(0, x.shape[1] - 1)[:, None])[:, 0]
    lp = torch.where(lp == NEG, lp, lp - torch.where(empty, torch.zeros_like(lse), lse))
    lp = torch.where(t >= x.shape[1], torch.full_like(lp, math.nan), lp)
    nan = torch.full_like(lse, math.nan)
    lp = torch.where(bad, nan, lp)
    lp = torch.where(t < 0, torch.zeros_like(lp), lp)
    lse, entropy = torch.where(bad, nan, lse), torch.where(bad, nan, entropy)
    value, ids = torch.sort(torch.nan_to_num(y, nan=NEG, posinf=NEG, neginf=NEG), dim=1, descending=True, stable=True)
    value, ids = value[:, :top_k], ids[:, :top_k]
    pad = top_k - value.shape[1]
    if pad > 0:
        value = torch.cat([value, torch.full((len(x), pad), NEG, dtype=value.dtype)], 1)
        ids = torch.cat([ids, torch.full((len(x), pad), -1)], 1)
    top = torch.where(value == NEG, value, value - torch.where(empty, torch.zeros_like(lse), lse)[:, None])
    ids = torch.where((value == NEG) | bad[:, None], torch.full_like(ids, -1), ids)
    top = torch.where(bad[:, None], nan[:, None], top)
    return {"logprobs": lp, "entropy": entropy, "logsumexp": lse, "top_logprobs": top, "top_ids": ids}


def close(got, want, tol):
    got = got.detach().cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isinf(got), torch.isinf(want)) and torch.equal(got[torch.isinf(got)], want[torch.isinf(want)])
    fine = torch.isfinite(want)
    off = (got - want).abs()[fine]
    assert bool((off <= (tol[fine] if isinstance(tol, torch.Tensor) else tol)).all()), off.max()


def check(logits, targets, top_k=0, temperature=1.0, **kw):
    r = ewg.token_logprobs(logits, targets, top_k=top_k, temperature=temperature, **kw)
    flat = logits.reshape(-1, logits.shape[-1])
    w = reference(flat, targets.reshape(-1), top_k, temperature)
    base = (flat.shape[1] / 256 + 64) * 2.0 ** -23
    for name in ("logprobs", "entropy", "logsumexp"):
        got = getattr(r, name)
        assert got.shape == targets.shape and got.dtype == torch.float32
        want = w[name]
        # the entropy weighs every distance with its probability: at most (1 + H) of the same
        close(got.reshape(-1), want, (1 + want.abs().nan_to_num(nan=0, posinf=0, neginf=0)) * base)
    if top_k:
        assert torch.equal(r.top_ids.reshape(-1, top_k).cpu(), w["top_ids"])
        want = w["top_logprobs"]
        close(r.top_logprobs.reshape(-1, top_k), want, (1 + want.abs().nan_to_num(nan=0, posinf=0, neginf=0)) * base)
    return r


def make(rows, vocab, dtype, seed, sigma=3.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=g) * sigma).to(dtype)
    t = torch.randint(0, vocab, (rows,), generator=g)
    return x.cuda(), t.cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,top_k", [
    (1, 1, 1), (3, 2, 5), (5, 7, 3), (2, 63, 32), (4, 255, 8), (1, 256, 4), (3, 257, 32), (2, 511, 5), (7, 513, 1),
    (1, 2048, 20), (2, 2049, 32), (1, 32003, 32), (33, 5003, 8), (3, 129280, 20), (1500, 1031, 3), (1, 262147, 7)])
def test_forward_sizes(dtype, rows, vocab, top_k):
    x, t = make(rows, vocab, dtype, rows * 7 + vocab)
    check(x, t, top_k)
    check(x, t.int(), 0, temperature=0.6)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [1, 3, 5])
def test_forward_any_element_alignment(dtype, offset):
    """Rows that start anywhere in 16 bytes, padded strides, and a transposed layout."""
    g = torch.Generator().manual_seed(offset)
    big = torch.randn(9, 1203, generator=g).to(dtype).cuda()
    x = big[:, offset:offset + 1111]
    t = torch.randint(0, 1111, (9,), generator=g).cuda()
    check(x, t, 6)
    check(big.t().contiguous().t()[:, offset:], t, 6)
    check(big[:8, :1200].reshape(2, 4, 1200)[:, :, offset:], t[:8].reshape(2, 4), 4)
    check(big[:1].expand(5, 1203), t[:5], 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [40, 515, 9001])
def test_masks_and_edges(dtype, vocab):
    lowest = torch.finfo(dtype).min
    x, t = make(16, vocab, dtype, vocab)
    x[0] = NEG                                   # nothing left
    x[1] = lowest                                # nothing left, by the type's lowest value
    x[2] = NEG
    x[2, vocab // 2] = -40.0                     # one token left
    t[2] = vocab // 2
    x[3, ::2] = NEG
    t[3] = 2                                     # a masked target
    x[4, 1::3] = lowest
    x[5, 5] = math.nan
    x[6, 7] = math.inf
    x[7] = math.nan
    t[7] = -1
    t[8] = -100                                  # no target
    t[9] = vocab                                 # beyond the vocabulary
    x[10] = 0.0                                  # all equal
    x[11] = -1e9                                 # a finite mask everywhere: uniform
    x[12] = 30000.0
    x[12, 3] = 30016.0
    x[13] = NEG
    t[13] = -1
    x[14, : vocab // 2] = -1e9
    for k in (0, 1, 5, 32):
        check(x, t, k)
        check(x, t, k, temperature=1.7)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [2, 1200])
def test_ties_go_to_the_lowest_index(dtype, rows):
    g = torch.Generator().manual_seed(rows)
    x = torch.randint(-2, 3, (rows, 3001), generator=g).to(dtype).cuda()
    x[0] = 1.0
    x[1] = -0.0
    x[1, 1::2] = 0.0                             # equal to -0
    t = torch.randint(0, 3001, (rows,), generator=g).cuda()
    check(x, t, 32)
    # ascending and descending rows: all of the largest in one group
    x[0] = torch.arange(3001).to(dtype).cuda() / 64
    x[1] = -x[0]
    check(x[:2].contiguous(), t[:2], 32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [1, 3, 700])
def test_many_large_logits_in_few_places(dtype, rows):
    """More candidates than are ranked at once: thousands of distinct large logits in a
    tenth of the lanes or of the groups, and thousands equal to the last one wanted."""
    vocab, size = 40000, 8 if dtype == torch.bfloat16 else 4               # elements of a 16-byte piece
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, vocab, generator=g)
    at = torch.arange(vocab)
    large = 50 + torch.randperm(vocab, generator=g).float() / 16
    x[0] = torch.where((at // size) % 64 < 6, large, x[0])                  # six lanes of every wave load
    if rows > 1:
        x[1] = torch.where((at // (16 * size)) % 64 < 6, large, x[1])       # six groups of every 64
        x[2] = -1e4                                                         # fewer allowed than wanted, a finite mask
        x[2, ::5000] = 3.0
    x = x.to(dtype).cuda()
    t = torch.randint(0, vocab, (rows,), generator=g).cuda()
    for k in (1, 20, 32):
        check(x[: min(rows, 3)].contiguous() if k < 20 else x, t[: min(rows, 3)] if k < 20 else t, k)


def test_splits_do_not_change_the_alternatives_and_calls_repeat():
    x, t = make(1, 129280, torch.bfloat16, 5)
    many = x.expand(2048, -1).contiguous()
    a = ewg.token_logprobs(x, t, top_k=32)
    b = ewg.token_logprobs(many, t.expand(2048).contiguous(), top_k=32)
    assert torch.equal(b.top_ids, a.top_ids.expand(2048, 32))
    assert bool((b.top_logprobs - a.top_logprobs).abs().max() <= 505 * 2.0 ** -23 * 16)
    again = ewg.token_logprobs(x, t, top_k=32)
    for u, v in zip(a, again):
        assert torch.equal(u, v)


def test_rows_beyond_32_bits_of_offset():
    """The last row starts past 2^32 bytes and past 2^31 elements."""
    rows, vocab = 70000, 31001
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(3)
    last = torch.randn(2, vocab, generator=g).bfloat16().cuda()
    x[-1], x[0] = last[0], last[1]
    t = torch.full((rows,), 17, dtype=torch.int64, device="cuda")
    r = ewg.token_logprobs(x, t, top_k=3)
    w = reference(last, torch.tensor([17, 17]), 3, 1.0)
    base = (vocab / 256 + 64) * 2.0 ** -23 * 16
    close(r.logprobs[[-1, 0]], w["logprobs"], base)
    assert torch.equal(r.top_ids[[-1, 0]].cpu(), w["top_ids"])
    assert bool((r.logprobs[1:-1] + math.log(vocab)).abs().max() < base)
    gl = torch.zeros(rows, device="cuda")
    gl[-1] = 2.0
    d = ewg.token_logprobs_backward(x, t, r.logsumexp, grad_logprobs=gl, out=x)
    want = 2.0 * (torch.nn.functional.one_hot(torch.tensor(17), vocab) - torch.softmax(last[0].cpu().double(), 0))
    close(d[-1], want, 2.0 ** -8 * want.abs() + 1e-6)
    assert int(torch.count_nonzero(d[1:-1])) == 0


# ---- backward -----------------------------------------------------------------

def backward_reference(logits, targets, lse, entropy, g, h, temperature):
    x = logits.cpu().double()
    y = torch.where(x <= -1e38, torch.full_like(x, NEG), x) / temperature
    lse, t = lse.cpu().double(), targets.cpu().long()
    empty = lse == NEG
    logp = y - torch.where(empty, torch.zeros_like(lse), lse)[:, None]
    p = torch.exp(logp)
    one = torch.zeros_like(p)
    ok = (t >= 0) & (t < x.shape[1])
    one[ok.nonzero()[:, 0], t[ok]] = 1
    g = torch.zeros(len(x)) if g is None else g.cpu()
    g = torch.where(t < 0, 0.0, g.double())
    h = (torch.zeros(len(x)) if h is None else h.cpu()).double()
    inner = torch.where(p == 0, torch.zeros_like(p), logp) + entropy.cpu().double()[:, None]
    d = (g[:, None] * (one - p) - h[:, None] * p * inner) / temperature
    d[empty] = 0
    d[t >= x.shape[1]] = math.nan
    size = (g.abs()[:, None] * p + h.abs()[:, None] * p * (inner.abs() + logp.abs().nan_to_num(nan=0, posinf=0, neginf=0))) / temperature
    tol = size * (8 + lse.abs().nan_to_num(nan=0, posinf=0, neginf=0))[:, None] * 2.0 ** -22 + 1e-37
    return d, tol + d.abs().nan_to_num(0) * (2.0 ** -8 if logits.dtype == torch.bfloat16 else 2.0 ** -21)


def check_backward(x, t, temperature=1.0, entropy=True, logprobs=True, out=None, seed=0):
    flat, tf = x.reshape(-1, x.shape[-1]), t.reshape(-1)
    g = torch.Generator().manual_seed(seed)
    gl = torch.randn(t.shape, generator=g).cuda() if logprobs else None
    gh = torch.randn(t.shape, generator=g).cuda() if entropy else None
    f = ewg.token_logprobs(x, t, temperature=temperature)
    want, tol = backward_reference(flat, tf, f.logsumexp.reshape(-1), f.entropy.reshape(-1),
                                   gl.reshape(-1) if logprobs else None, gh.reshape(-1) if entropy else None, temperature)
    d = ewg.token_logprobs_backward(x, t, f.logsumexp, f.entropy if entropy else None, gl, gh, temperature, out=out)
    assert d.shape == x.shape and d.dtype == x.dtype
    close(d.reshape(-1, x.shape[-1]), want, tol)
    return d


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (5, 7), (2, 255), (4, 4096), (3, 4097), (2, 8193), (33, 5003), (1, 129280)])
@pytest.mark.parametrize("entropy", [False, True])
def test_backward_sizes(dtype, rows, vocab, entropy):
    x, t = make(rows, vocab, dtype, rows + vocab)
    check_backward(x, t, entropy=entropy)
    check_backward(x, t.int(), 0.8, entropy=True, logprobs=entropy)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward_layouts(dtype):
    g = torch.Generator().manual_seed(1)
    big = torch.randn(8, 1203, generator=g).to(dtype).cuda()
    t = torch.randint(0, 1100, (8,), generator=g).cuda()
    x = big[:, 3:1103]
    check_backward(x, t)                                               # rows and result at different offsets
    out = torch.full_like(big, 7.0)
    d = check_backward(x, t, out=out[:, 3:1103])                       # the same offsets, padded
    assert d.data_ptr() == out[:, 3:].data_ptr()
    assert bool((out[:, :3] == 7).all()) and bool((out[:, 1103:] == 7).all())
    check_backward(big[:, :1200].reshape(2, 4, 1200), t.reshape(2, 4))
    y = x.contiguous()
    want = ewg.token_logprobs_backward(y, t, ewg.token_logprobs(y, t).logsumexp, grad_logprobs=torch.ones(8, device="cuda"))
    lse = ewg.token_logprobs(y, t).logsumexp
    assert ewg.token_logprobs_backward(y, t, lse, grad_logprobs=torch.ones(8, device="cuda"), out=y) is y
    assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward_masks_and_edges(dtype):
    x, t = make(10, 777, dtype, 4)
    x[0] = NEG
    x[1] = torch.finfo(dtype).min
    x[2, 1:] = NEG
    t[2] = 0
    x[3, ::2] = NEG
    t[3] = 4
    x[4, ::3] = torch.finfo(dtype).min
    t[5] = -100
    t[6] = 777
    check_backward(x, t)
    check_backward(x, t, entropy=False)
    x[7, 9] = math.nan
    lse = ewg.token_logprobs(x, t)
    d = ewg.token_logprobs_backward(x, t, lse.logsumexp, lse.entropy, torch.ones(10, device="cuda"))
    assert bool(torch.isnan(d[7]).all()) and not bool(torch.isnan(d[:6]).any())


@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_backward_matches_differences(temperature):
    """The gradient of a weighted sum of log probabilities and entropies, against central
    differences of the 64-bit definition: the step 1e-5 leaves 1e-9 of curvature and
    rounding, far below the kernel's own 32-bit error."""
    x, t = make(3, 17, torch.float32, 8, sigma=1.5)
    gl = torch.tensor([0.7, -1.3, 0.4], device="cuda")
    gh = torch.tensor([-0.2, 0.9, 1.1], device="cuda")
    f = ewg.token_logprobs(x, t, temperature=temperature)
    d = ewg.token_logprobs_backward(x, t, f.logsumexp, f.entropy, gl, gh, temperature).cpu().double()

    def value(z):
        logp = torch.log_softmax(z / temperature, 1)
        return (gl.cpu().double() * logp.gather(1, t.cpu()[:, None])[:, 0]).sum() \
            + (gh.cpu().double() * -(logp.exp() * logp).sum(1)).sum()

    z = x.cpu().double()
    for i in range(3):
        for j in range(17):
            up, down = z.clone(), z.clone()
            up[i, j] += 1e-5
            down[i, j] -= 1e-5
            assert abs((value(up) - value(down)) / 2e-5 - d[i, j]) < 4e-6


# ---- streams, graphs, refusals ---------------------------------------------------

def test_runs_on_the_current_stream_and_in_a_graph():
    x, t = make(5, 40000, torch.bfloat16, 6)
    want = ewg.token_logprobs(x, t, top_k=4)
    gl = torch.ones(5, device="cuda")
    grad = ewg.token_logprobs_backward(x, t, want.logsumexp, grad_logprobs=gl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ewg.token_logprobs(x, t, top_k=4)
    torch.cuda.current_stream().wait_stream(side)
    for u, v in zip(got, want):
        assert torch.equal(u, v)
    ws = torch.empty(max(1, ewg.token_logprobs_workspace_bytes(5, 40000, torch.bfloat16, 4)), dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(side):
        ewg.token_logprobs(x, t, top_k=4, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = ewg.token_logprobs(x, t, top_k=4, workspace=ws)
        d = ewg.token_logprobs_backward(x, t, r.logsumexp, grad_logprobs=gl)
    for i in range(3):
        x.copy_(make(5, 40000, torch.bfloat16, 60 + i)[0])
        graph.replay()
        torch.cuda.synchronize()
        e = ewg.token_logprobs(x, t, top_k=4)
        for u, v in zip(r, e):
            assert torch.equal(u, v)
        assert torch.equal(d, ewg.token_logprobs_backward(x, t, e.logsumexp, grad_logprobs=gl))
    assert grad.shape == x.shape


def test_empty_and_refusals():
    x, t = make(4, 100, torch.bfloat16, 1)
    e = ewg.token_logprobs(x[:0], t[:0], top_k=3)
    assert e.logprobs.shape == (0,) and e.top_ids.shape == (0, 3)
    assert ewg.token_logprobs_backward(x[:0], t[:0], e.logsumexp).shape == (0, 100)
    lse = ewg.token_logprobs(x, t).logsumexp
    one = torch.ones(4, device="cuda")
    for bad in (lambda: ewg.token_logprobs(x.half(), t), lambda: ewg.token_logprobs(x, t.short()),
                lambda: ewg.token_logprobs(x, t[:3]), lambda: ewg.token_logprobs(x.cpu(), t),
                lambda: ewg.token_logprobs(x, t, top_k=33), lambda: ewg.token_logprobs(x, t, top_k=-1),
                lambda: ewg.token_logprobs(x, t, temperature=0.0), lambda: ewg.token_logprobs(x, t, temperature=math.nan),
                lambda: ewg.token_logprobs(x[:, :0], t), lambda: ewg.token_logprobs(x, None),
                lambda: ewg.token_logprobs(x, t, workspace=torch.empty(9, device="cuda")),
                lambda: ewg.token_logprobs_backward(x, t, lse[:3]),
                lambda: ewg.token_logprobs_backward(x, t, lse.double()),
                lambda: ewg.token_logprobs_backward(x, t, lse, None, one, one),
                lambda: ewg.token_logprobs_backward(x, t, lse, None, one, out=x.float()),
                lambda: ewg.token_logprobs_backward(x, t, lse, None, one, out=torch.empty(100, 4, dtype=x.dtype, device="cuda").t())):
        with pytest.raises(ValueError):
            bad()
