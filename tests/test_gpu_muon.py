"""orthogonalize_update and muon_step against the definitions in 64 bits.

Tolerance. Each step rounds its copies of X, A and B to half precision (2^-12 of an
entry, independent of each other); through B = bA + cAA and B X that is at most
(|a| + |b| + |c|) 2^-12 = 0.25 % of the norm a step, and the steps map all but the
smallest singular values onto a bounded range, so errors of earlier steps do not add
up: twice one step's, 5e-3 of the result's norm, holds for any number of steps up to
five. A bfloat16 result adds 2^-9.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

import sparse_embedding_weight_amd as ewg  # noqa: E402

TOL = 5e-3
BF16 = 2.0 ** -9


@pytest.fixture(autouse=True)
def _gpu(require_gpu):
    yield


def reference(u, steps=5, coefficients=ewg.NEWTON_SCHULZ_COEFFICIENTS, eps=1e-7):
    x = u.detach().cpu().double()
    if x.shape[-2] > x.shape[-1]:
        return reference(x.transpose(-2, -1), steps, coefficients, eps).transpose(-2, -1)
    x = x / (x.flatten(-2).norm(dim=-1)[..., None, None] + eps)
    a, b, c = coefficients
    for _ in range(steps):
        y = x @ x.transpose(-2, -1)
        x = a * x + (b * y + c * y @ y) @ x
    return x


def off(got, want):
    got = got.detach().cpu().double()
    return float(((got - want).flatten(-2).norm(dim=-1) / want.flatten(-2).norm(dim=-1).clamp(min=1e-300)).max())


def make(shape, dtype, seed, rank=0, scale=1e-3):
    g = torch.Generator().manual_seed(seed)
    u = torch.randn(shape, generator=g)
    if rank:
        u = 0.05 * u + torch.randn(*shape[:-1], rank, generator=g) @ torch.randn(*shape[:-2], rank, shape[-1], generator=g)
    return (u * scale).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (9, 1), (2, 3), (31, 33), (64, 64), (65, 64), (127, 129), (128, 128),
                                   (129, 500), (777, 130), (256, 1031), (3, 5, 11), (4, 130, 70), (7, 64, 192)])
def test_orthogonalize_sizes(dtype, shape):
    u = make(shape, dtype, sum(shape))
    assert off(ewg.orthogonalize_update(u), reference(u)) < TOL + BF16


@pytest.mark.parametrize("shape", [(2048, 2050), (2300, 2111), (520, 4100)])
def test_orthogonalize_large(shape):
    u = make(shape, torch.float32, 11, rank=40)
    want = reference(u.cpu())
    assert off(ewg.orthogonalize_update(u), want) < TOL + BF16


@pytest.mark.parametrize("shape", [(40, 200, 260), (300, 170, 150), (3, 1300, 1500), (2500, 2700), (2700, 2500), (4096, 1024),
                                   (8, 700, 900), (64, 310, 300), (2, 2304, 2304), (100, 256, 512), (6530, 6600)])
def test_every_tile_size(shape):
    """Sizes and batches for which the products take each of their tiles, alone and in
    pairs, with partly filled last tiles; the reference in 64 bits on the GPU."""
    u = make(shape, torch.bfloat16, 21, rank=20)

    def on_gpu(x):
        if x.shape[-2] > x.shape[-1]:
            return on_gpu(x.transpose(-2, -1).contiguous()).transpose(-2, -1)
        x = x / (x.flatten(-2).norm(dim=-1)[..., None, None] + 1e-7)
        a, b, c = ewg.NEWTON_SCHULZ_COEFFICIENTS
        for _ in range(5):
            y = x @ x.transpose(-2, -1).contiguous()
            x = a * x + (b * y + c * (y @ y)) @ x
        return x

    want = on_gpu(u.double()).cpu()
    assert off(ewg.orthogonalize_update(u), want) < TOL + BF16
    w, m = torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
    ewg.muon_step(w, u, m, lr=1.0, beta=0.5, nesterov=False, scale=1.0)      # weight = -result, in 32 bits
    assert off(-w, want) < TOL
    assert torch.equal(m, u.float())


@pytest.mark.parametrize("rank", [1, 4, 30])
def test_orthogonalize_strong_directions_over_noise(rank):
    u = make((240, 300), torch.float32, rank, rank=rank)
    assert off(ewg.orthogonalize_update(u), reference(u)) < TOL + BF16


@pytest.mark.parametrize("steps,coefficients", [(1, (3.4445, -4.7750, 2.0315)), (3, (2.0, -1.5, 0.5)), (8, (1.875, -1.25, 0.375))])
def test_steps_and_coefficients(steps, coefficients):
    u = make((90, 140), torch.float32, 2)
    got = ewg.orthogonalize_update(u, steps=steps, coefficients=coefficients)
    assert off(got, reference(u, steps, coefficients)) < TOL + BF16


def test_scale_of_the_update_does_not_matter():
    """1e-24 and 1e+24: squares outside 32 bits."""
    u = make((70, 90), torch.float32, 3, scale=1.0)
    want = reference(u, eps=0.0)
    for s in (1e-24, 1.0, 1e24):
        assert off(ewg.orthogonalize_update(u * s, eps=0.0), want) < TOL + BF16
    one = torch.zeros(50, 60, device="cuda")
    one[3, 5] = 1e-12                            # eps far above the norm
    assert off(ewg.orthogonalize_update(one), reference(one)) < TOL + BF16


def test_zero_nan_and_inf():
    u = make((4, 100, 60), torch.float32, 4)
    u[1] = 0
    u[2, 5, 5] = math.nan
    u[3, 7, 7] = math.inf
    got = ewg.orthogonalize_update(u)
    assert int(torch.count_nonzero(got[1])) == 0
    assert bool(torch.isnan(got[2]).all()) and bool(torch.isnan(got[3]).all())
    assert off(got[0], reference(u[0])) < TOL + BF16          # neighbours keep theirs


def test_layouts_and_in_place():
    g = torch.Generator().manual_seed(5)
    big = torch.randn(3, 200, 301, generator=g).bfloat16().cuda()
    u = big[:, 10:150, 7:240]
    want = reference(u)
    assert off(ewg.orthogonalize_update(u), want) < TOL + BF16
    out = torch.full_like(big, 9.0)
    ewg.orthogonalize_update(u, out=out[:, 10:150, 7:240])
    assert off(out[:, 10:150, 7:240], want) < TOL + BF16
    out[:, 10:150, 7:240] = 9.0
    assert bool((out == 9.0).all())
    same = ewg.orthogonalize_update(u)
    assert ewg.orthogonalize_update(u, out=u) is u
    assert torch.equal(u, same)


def test_repeats_bit_for_bit_on_streams_and_in_a_graph():
    u = make((2, 260, 390), torch.bfloat16, 6)
    want = ewg.orthogonalize_update(u)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ewg.orthogonalize_update(u)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    ws = torch.empty(ewg.orthogonalize_update_workspace_bytes(2, 260, 390), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = ewg.orthogonalize_update(u, workspace=ws)
    for i in range(3):
        u.copy_(make((2, 260, 390), torch.bfloat16, 60 + i))
        ws.fill_(0xff)                           # what the workspace held does not matter
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r, ewg.orthogonalize_update(u))


@pytest.mark.parametrize("weight_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("grad_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape,nesterov", [((70, 130), True), ((259, 64), False), ((3, 40, 41), True)])
def test_muon_step(weight_dtype, grad_dtype, shape, nesterov):
    w = make(shape, weight_dtype, 1, scale=0.02)
    g = make(shape, grad_dtype, 2)
    m = make(shape, torch.float32, 3, scale=4e-3)
    lr, beta, decay, scale = 2e-2, 0.9, 0.1, 1.7
    want_m = beta * m.cpu().double() + g.cpu().double()
    o = reference(g.cpu().double() + beta * want_m if nesterov else want_m)
    want_w = w.cpu().double() * (1 - lr * decay) - lr * scale * o
    new_w, new_m = torch.empty_like(w), torch.empty_like(m)
    old_w, old_m = w.clone(), m.clone()
    kw = dict(lr=lr, beta=beta, nesterov=nesterov, weight_decay=decay, scale=scale)
    ewg.muon_step(w, g, m, out_weight=new_w, out_momentum=new_m, **kw)
    assert torch.equal(w, old_w) and torch.equal(m, old_m)
    assert off(new_m, want_m) < 2.0 ** -22
    size = (want_w.norm() + TOL / 2.0 ** -23 * lr * scale * o.norm() * 2.0 ** -23 / TOL).item()
    err = (new_w.cpu().double() - want_w).norm().item()
    rounding = BF16 if weight_dtype == torch.bfloat16 else 2.0 ** -22
    assert err <= rounding * size + TOL * lr * scale * o.norm().item()
    ewg.muon_step(w, g, m, **kw)                 # in place: the same bits
    assert torch.equal(w, new_w) and torch.equal(m, new_m)


def test_muon_step_default_scale_and_padded_strides():
    big = make((2, 90, 64), torch.float32, 8, scale=0.02)
    w, g, m = big[:, :80, :33], make((2, 80, 40), torch.bfloat16, 9)[:, :, 5:38], torch.zeros(2, 81, 35, device="cuda")[:, 1:, 1:34]
    rest = big.clone()
    want = w.cpu().double() - 0.01 * math.sqrt(80 / 33) * reference(g.cpu().double())
    ewg.muon_step(w, g, m, lr=0.01, nesterov=False)
    assert float((w.cpu().double() - want).norm()) < TOL * 0.01 * math.sqrt(80 / 33) * math.sqrt(66) * 1.3
    assert torch.equal(m, g.float())
    big[:, :80, :33] = rest[:, :80, :33]
    assert torch.equal(big, rest)


def test_empty_and_refusals():
    assert ewg.orthogonalize_update(torch.empty(0, 5, device="cuda")).shape == (0, 5)
    assert ewg.orthogonalize_update(torch.empty(0, 4, 5, device="cuda")).shape == (0, 4, 5)
    u = make((8, 12), torch.float32, 1)
    w, m = u.clone(), u.clone()
    for bad in (lambda: ewg.orthogonalize_update(u.half()), lambda: ewg.orthogonalize_update(u.cpu()),
                lambda: ewg.orthogonalize_update(u[0]), lambda: ewg.orthogonalize_update(u.t()),
                lambda: ewg.orthogonalize_update(u[:1].expand(8, 12)), lambda: ewg.orthogonalize_update(u, steps=0),
                lambda: ewg.orthogonalize_update(u, steps=65), lambda: ewg.orthogonalize_update(u, eps=-1.0),
                lambda: ewg.orthogonalize_update(u, coefficients=(1.0, math.nan, 0.0)),
                lambda: ewg.orthogonalize_update(u, out=torch.empty_like(u)),
                lambda: ewg.orthogonalize_update(u, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
                lambda: ewg.orthogonalize_update(torch.empty(1, 40000, device="cuda")),
                lambda: ewg.muon_step(w, u[:4], m, lr=0.1), lambda: ewg.muon_step(w, u, m.bfloat16(), lr=0.1),
                lambda: ewg.muon_step(w, u.half(), m, lr=0.1), lambda: ewg.muon_step(w, u, m.cpu(), lr=0.1),
                lambda: ewg.muon_step(w, u, m, lr=0.1, out_weight=w.bfloat16()),
                lambda: ewg.muon_step(w, u, m, lr=0.1, out_momentum=torch.empty(8, 24, device="cuda")[:, :12])):
        with pytest.raises(ValueError):
            bad()
