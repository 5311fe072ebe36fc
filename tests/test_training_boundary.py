"""Host-side tests of the C entry points of include/token_logprobs.h and
include/muon.h (no GPU work): constants, workspace sizes, and argument errors that
return before anything is enqueued; the same once more with the library's host
code under AddressSanitizer. Gradients of the documented formulas against
differences, in 64 bits."""
import math
import os
import re
import subprocess
import sys

import pytest
import torch

import sparse_embedding_weight_amd as ewg
from sparse_embedding_weight_amd import _binding as B
from sparse_embedding_weight_amd import _logprobs as L
from sparse_embedding_weight_amd import _muon as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALLS = r'''
OK, UNSUPPORTED, INVALID, WS_SMALL = 0, 1, 2, 3
I32, I64, BF16, F32 = 0, 1, 2, 3
HUGE = 1 << 62

def forward(f, **kw):
    a = dict(logits=64, targets=64, rows=4, vocab=100, stride=100, dt=BF16, tt=I64, temp=1.0, k=3, lp=64, en=64,
             lse=64, top=64, ids=64, ws=256, wsb=1 << 30)
    a.update(kw)
    return f(a["logits"], a["targets"], a["rows"], a["vocab"], a["stride"], a["dt"], a["tt"], a["temp"], a["k"],
             a["lp"], a["en"], a["lse"], a["top"], a["ids"], a["ws"], a["wsb"], None)

def backward(f, **kw):
    a = dict(logits=64, targets=64, lse=64, en=64, g=64, h=64, out=64, rows=4, vocab=100, stride=100, ostride=100,
             dt=BF16, tt=I64, temp=1.0)
    a.update(kw)
    return f(a["logits"], a["targets"], a["lse"], a["en"], a["g"], a["h"], a["out"], a["rows"], a["vocab"], a["stride"],
             a["ostride"], a["dt"], a["tt"], a["temp"], None)

def ortho(f, **kw):
    a = dict(u=64, out=64, batch=2, rows=8, cols=16, ub=128, ur=16, ob=128, orow=16, dt=F32, steps=5, a=3.4, b=-4.7,
             c=2.0, eps=1e-7, ws=256, wsb=1 << 40)
    a.update(kw)
    return f(a["u"], a["out"], a["batch"], a["rows"], a["cols"], a["ub"], a["ur"], a["ob"], a["orow"], a["dt"],
             a["steps"], a["a"], a["b"], a["c"], a["eps"], a["ws"], a["wsb"], None)

def muon(f, **kw):
    a = dict(w=64, ow=64, g=64, m=64, om=64, batch=2, rows=8, cols=16, wb=128, wr=16, gb=128, gr=16, mb=128, mr=16,
             wd=BF16, gd=F32, lr=0.1, beta=0.9, nest=1, decay=0.0, scale=1.0, steps=5, a=3.4, b=-4.7, c=2.0, eps=1e-7,
             ws=256, wsb=1 << 40)
    a.update(kw)
    return f(a["w"], a["ow"], a["g"], a["m"], a["om"], a["batch"], a["rows"], a["cols"], a["wb"], a["wr"], a["gb"],
             a["gr"], a["mb"], a["mr"], a["wd"], a["gd"], a["lr"], a["beta"], a["nest"], a["decay"], a["scale"],
             a["steps"], a["a"], a["b"], a["c"], a["eps"], a["ws"], a["wsb"], None)

def check(lib):
    nan, inf = float("nan"), float("inf")
    f = lib.token_logprobs
    assert forward(f, rows=0) == OK and forward(f, rows=0, logits=None, targets=None, lp=None) == OK
    for bad in (dict(dt=9), dict(tt=-1), dict(temp=0.0), dict(temp=nan), dict(temp=inf), dict(temp=-1.0), dict(stride=99),
                dict(logits=None), dict(targets=None), dict(lp=None), dict(en=None), dict(lse=None), dict(top=None),
                dict(ids=None), dict(logits=65), dict(dt=F32, logits=66), dict(vocab=20000, stride=20000, ws=None),
                dict(vocab=20000, stride=20000, ws=264)):
        assert forward(f, **bad) == INVALID, bad
    for bad in (dict(dt=I32), dict(tt=F32), dict(rows=-1), dict(rows=(1 << 20) + 1), dict(vocab=0), dict(vocab=-4),
                dict(vocab=(1 << 20) + 1, stride=HUGE), dict(rows=HUGE), dict(k=33), dict(k=-1)):
        assert forward(f, **bad) == UNSUPPORTED, bad
    size = lib.token_logprobs_workspace_bytes
    need = size(4, 20000, BF16, 3)
    assert need > 0 and forward(f, vocab=20000, stride=20000, wsb=need - 1) == WS_SMALL
    assert size(4, 100, BF16, 3) == 0 and size(4096, 129280, BF16, 0) == 0
    for args in ((0, 100, BF16, 0), (-1, 100, BF16, 0), (4, 0, BF16, 0), (4, HUGE, BF16, 0), (4, 100, I32, 0), (4, 100, F32, 33)):
        assert size(*args) == 0
    for rows in (1, 7, 511, 512, 1 << 20):
        for vocab in (1, 2, 4096, 129280, 1 << 20):
            for dt in (BF16, F32):
                assert size(rows, vocab, dt, 32) >= size(rows, vocab, dt, 0) >= 0
    f = lib.token_logprobs_backward
    assert backward(f, rows=0) == OK
    for bad in (dict(dt=77), dict(temp=nan), dict(stride=99), dict(ostride=99), dict(logits=None), dict(targets=None),
                dict(lse=None), dict(out=None), dict(en=None), dict(out=65), dict(logits=65)):
        assert backward(f, **bad) == INVALID, bad
    for bad in (dict(dt=I64), dict(tt=BF16), dict(rows=-3), dict(vocab=0), dict(vocab=HUGE)):
        assert backward(f, **bad) == UNSUPPORTED, bad
    f = lib.orthogonalize_update
    assert ortho(f, batch=0) == OK and ortho(f, rows=0) == OK and ortho(f, cols=0, u=None) == OK
    for bad in (dict(dt=9), dict(eps=-1.0), dict(eps=nan), dict(a=nan), dict(b=inf), dict(c=nan), dict(u=None), dict(out=None),
                dict(ur=15), dict(orow=15), dict(ub=127), dict(ob=0), dict(ws=None), dict(ws=300)):
        assert ortho(f, **bad) == INVALID, bad
    for bad in (dict(dt=I32), dict(steps=0), dict(steps=65), dict(rows=32769), dict(cols=HUGE), dict(batch=65536), dict(rows=-1),
                dict(batch=-1)):
        assert ortho(f, **bad) == UNSUPPORTED, bad
    size = lib.orthogonalize_update_workspace_bytes
    need = size(2, 8, 16)
    assert need > 0 and ortho(f, wsb=need - 1) == WS_SMALL
    assert size(0, 8, 8) == 0 and size(1, 32769, 1) == 0 and size(1, -1, 4) == 0 and size(HUGE, 4, 4) == 0
    assert size(1, 100, 7000) == size(1, 7000, 100) and size(65535, 32768, 32768) > 1 << 46
    f = lib.muon_step
    assert muon(f, batch=0) == OK and muon(f, cols=0) == OK
    for bad in (dict(wd=9), dict(gd=-1), dict(nest=2), dict(eps=nan), dict(w=None), dict(ow=None), dict(g=None), dict(m=None),
                dict(om=None), dict(wr=15), dict(gb=10), dict(mr=15), dict(ws=None), dict(ws=257)):
        assert muon(f, **bad) == INVALID, bad
    for bad in (dict(wd=I32), dict(gd=I64), dict(steps=0), dict(rows=32769)):
        assert muon(f, **bad) == UNSUPPORTED, bad
    assert muon(f, wsb=need - 1) == WS_SMALL
'''

ASAN = r'''
import ctypes, sys
lib = ctypes.CDLL(sys.argv[1])
i64, i32, vp, sz, f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
def sig(name, args, res=i32):
    f = getattr(lib, name); f.argtypes = args; f.restype = res
sig("token_logprobs_workspace_bytes", [i64, i64, i32, i32], sz)
sig("token_logprobs", [vp, vp, i64, i64, i64, i32, i32, f32, i32] + [vp] * 6 + [sz, vp])
sig("token_logprobs_backward", [vp] * 7 + [i64] * 4 + [i32, i32, f32, vp])
sig("orthogonalize_update_workspace_bytes", [i64] * 3, sz)
sig("orthogonalize_update", [vp, vp] + [i64] * 7 + [i32, i32] + [f32] * 4 + [vp, sz, vp])
sig("muon_step", [vp] * 5 + [i64] * 9 + [i32, i32, f32, f32, i32, f32, f32, i32] + [f32] * 4 + [vp, sz, vp])
''' + CALLS + '\ncheck(lib)\nprint("host checks ok")\n'


def test_argument_errors_return_before_any_launch():
    space = {}
    exec(CALLS, space)
    space["check"](B.lib)


def test_host_entry_points_under_address_sanitizer():
    sys.path.insert(0, os.path.join(ROOT, "sparse_embedding_weight_amd"))
    import build
    runtime = build.asan_runtime()
    if not runtime:
        pytest.skip("the compiler's shared AddressSanitizer runtime is not installed")
    env = dict(os.environ, LD_PRELOAD=runtime, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1")
    r = subprocess.run([sys.executable, "-c", ASAN, build.build_host_asan()], capture_output=True, text=True, env=env, timeout=300)
    assert "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
    assert r.returncode == 0 and "host checks ok" in r.stdout, r.stderr[-4000:]


def test_constants_match_the_headers():
    text = "".join(open(os.path.join(ROOT, "include", n)).read() for n in ("token_logprobs.h", "muon.h"))
    c = {k: int(v) for k, v in re.findall(r"^#define\s+(EWG_\w+)\s+(\d+)\s*$", text, flags=re.M)}
    assert c == {"EWG_MAX_TOP_LOGPROBS": ewg.MAX_TOP_LOGPROBS, "EWG_LOGPROBS_MAX_ROWS": L.MAX_ROWS,
                 "EWG_LOGPROBS_MAX_VOCAB": L.MAX_VOCAB, "EWG_MUON_MAX_SIDE": M.MAX_SIDE,
                 "EWG_MUON_MAX_BATCH": M.MAX_BATCH, "EWG_MUON_MAX_STEPS": M.MAX_STEPS}


def test_cpu_tensors_are_refused():
    with pytest.raises(ValueError):
        ewg.token_logprobs(torch.zeros(2, 3), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        ewg.orthogonalize_update(torch.zeros(2, 3))
    with pytest.raises(ValueError):
        ewg.muon_step(torch.zeros(2, 3), torch.zeros(2, 3), torch.zeros(2, 3), lr=0.1)


@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_gradient_formula_against_differences(temperature):
    """(g ([j = t] - p) - h p (ln p + H)) / T is the gradient of g logprob + h H: central
    differences of step 1e-5 agree within 1e-9 of curvature and 1e-10 of rounding."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(9, generator=g, dtype=torch.float64)
    t, gl, gh = 5, 0.8, -0.6

    def value(z):
        logp = torch.log_softmax(z / temperature, 0)
        return gl * logp[t] - gh * (logp.exp() * logp).sum()

    logp = torch.log_softmax(x / temperature, 0)
    p, entropy = logp.exp(), -(logp.exp() * logp).sum()
    one = torch.nn.functional.one_hot(torch.tensor(t), 9)
    formula = (gl * (one - p) - gh * p * (logp + entropy)) / temperature
    for j in range(9):
        e = torch.zeros(9, dtype=torch.float64)
        e[j] = 1e-5
        assert math.isclose(float(value(x + e) - value(x - e)) / 2e-5, float(formula[j]), rel_tol=0, abs_tol=2e-9)
