"""Arguments that the norm, gate and MoE layer entry points refuse, before any device
call, and the device and stream they run on (no GPU needed)."""
import contextlib
import ctypes
import types

import pytest
import torch
from torch.autograd import forward_ad

from moe_grouped_gemm_nvfp4_gb300 import fp8, gating, moe, norm, tokens
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)
TWO = ctypes.c_void_p(4098)
INV, UNS = F.NVFP4_ERR_INVALID_ARG, F.NVFP4_ERR_UNSUPPORTED


def test_norm_refusals():
    lib = F.load()

    def plain(x=P, ld=64, r=P, ldr=64, T=4, D=64, dt=0, w=P, wt=0, eps=1e-6, h=P, y=P):
        return lib.nvfp4_rms_norm(x, ld, r, ldr, T, D, dt, w, wt, eps, h, y, None)

    def codes(x=P, ld=64, r=P, ldr=64, T=4, D=64, dt=0, w=P, wt=0, eps=1e-6, h=P, q=P, s=P):
        return lib.nvfp4_rms_norm_fp8(x, ld, r, ldr, T, D, dt, w, wt, eps, h, q, s, None)

    def grad(dy=P, ldd=64, x=P, ld=64, r=P, ldr=64, T=4, D=64, dt=0, w=P, wt=0, eps=1e-6, dx=P,
             dw=P, ws=P, n=1 << 30):
        return lib.nvfp4_rms_norm_grad(dy, ldd, x, ld, r, ldr, T, D, dt, w, wt, eps, dx, dw, ws, n,
                                       None)

    nan = float("nan")
    for call in (plain, codes, grad):
        for bad in (dict(T=-1), dict(D=0), dict(dt=3), dict(wt=-1), dict(w=None), dict(eps=-1.0),
                    dict(eps=nan), dict(ld=63), dict(ldr=63), dict(x=None)):
            assert call(**bad) == INV, (call, bad)
        for bad in (dict(D=16400, ld=16400, ldr=16400, **({"ldd": 16400} if call is grad else {})),
                    dict(wt=1), dict(x=ODD), dict(w=ODD), dict(r=TWO)):
            assert call(**bad) == UNS, (call, bad)
    assert plain(h=None) == INV and plain(y=None) == INV and plain(r=None, h=None, y=None) == INV
    assert plain(y=TWO) == UNS and plain(ld=68) == UNS and plain(h=TWO) == UNS
    assert codes(q=None) == INV and codes(s=None) == INV and codes(h=None) == INV
    for bad in (dict(dt=2, wt=2), dict(D=56), dict(ld=68), dict(q=TWO), dict(w=TWO),
                dict(s=ctypes.c_void_p(4098))):
        assert codes(**bad) == UNS, bad
    for name in ("dy", "dx", "dw", "ws"):
        assert grad(**{name: None}) == INV
    assert grad(ldd=60) == INV and grad(ldd=68) == UNS and grad(dx=TWO) == UNS
    need = F.nvfp4_rms_norm_grad_workspace_bytes(4, 64)
    assert need > 0 and grad(n=need - 1) == UNS
    assert F.nvfp4_rms_norm_grad_workspace_bytes(0, 64) == 0
    assert F.nvfp4_rms_norm_grad_workspace_bytes(4, 0) == 0


def test_gate_refusals():
    lib = F.load()

    def gate(l=P, ld=8, T=4, E=8, dt=2, k=2, bias=None, flags=0, ids=P, w=P):
        return lib.nvfp4_topk_gate(l, ld, T, E, dt, k, bias, flags, 1.0, ids, w, None)

    def grad(dw=P, l=P, ld=8, T=4, E=8, dt=2, k=2, ids=P, flags=0, dl=P):
        return lib.nvfp4_topk_gate_grad(dw, l, ld, T, E, dt, k, ids, flags, 1.0, dl, None)

    for call in (gate, grad):
        for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(ld=7), dict(dt=4),
                    dict(flags=4), dict(l=None), dict(ids=None)):
            assert call(**bad) == INV, (call, bad)
        for bad in (dict(E=1025, ld=1025), dict(E=64, ld=64, k=33), dict(l=ODD), dict(ids=TWO)):
            assert call(**bad) == UNS, (call, bad)
    assert gate(w=None) == INV and gate(bias=TWO) == UNS
    assert grad(dw=None) == INV and grad(dl=None) == INV and grad(dl=TWO) == UNS


def test_layer_refusals():
    lib = F.load()
    need = F.nvfp4_fp8_moe_layer_workspace_bytes(4, 2, 8, 64, 32, 48)
    assert need > 0

    def layer(x=P, ld=64, T=4, dt=0, router=P, rt=0, bias=None, flags=0, W1=P, s1=P, W2=P, s2=P, E=8,
              k=2, K=64, I=32, N=48, ids=P, w=P, out=P, ldo=48, ws=P, n=need):
        return lib.nvfp4_fp8_moe_layer(x, ld, T, dt, router, rt, bias, flags, 1.0, W1, s1, W2, s2, E,
                                       k, K, I, N, ids, w, out, ldo, ws, n, None)

    for bad in (dict(T=-1), dict(dt=7), dict(rt=7), dict(E=0), dict(k=0), dict(k=9), dict(K=0),
                dict(I=0), dict(N=0), dict(ld=60), dict(ldo=47), dict(flags=8), dict(W1=None),
                dict(s1=None), dict(W2=None), dict(s2=None), dict(x=None), dict(ids=None),
                dict(w=None), dict(out=None), dict(ws=None), dict(router=None, bias=P),
                dict(router=None, flags=1)):
        assert layer(**bad) == INV, bad
    for bad in (dict(dt=2), dict(rt=1), dict(x=TWO), dict(router=TWO), dict(W1=TWO), dict(W2=TWO),
                dict(s1=TWO), dict(s2=TWO), dict(bias=TWO), dict(ids=TWO), dict(w=TWO), dict(out=ODD),
                dict(ws=TWO), dict(ld=68), dict(K=72, ld=72), dict(I=40), dict(T=9, n=1 << 40),
                dict(n=need - 1), dict(E=1025, n=1 << 40), dict(E=64, k=33, n=1 << 40),
                dict(N=(1 << 20) + 1, ldo=1 << 21, n=1 << 60)):
        assert layer(**bad) == UNS, bad
    for sizes in ((0, 2, 8, 64, 32, 48), (9, 2, 8, 64, 32, 48), (4, 9, 8, 64, 32, 48),
                  (4, 2, 0, 64, 32, 48), (4, 2, 8, 72, 32, 48), (4, 2, 8, 64, 40, 48),
                  (4, 2, 8, 64, 32, 0), (-1, 2, 8, 64, 32, 48)):
        assert F.nvfp4_fp8_moe_layer_workspace_bytes(*sizes) == 0


def test_python_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.ones(64)
    for bad in (lambda: norm.rms_norm(x, w[:32]), lambda: norm.rms_norm(x, w.half()),
                lambda: norm.rms_norm(x, w, x[:2]), lambda: norm.rms_norm(x, w, x.float()),
                lambda: norm.rms_norm(x.double(), w), lambda: norm.rms_norm(x, w, eps=-1.0),
                lambda: norm.rms_norm(torch.tensor(1.0), w), lambda: norm.rms_norm(x, w),
                lambda: norm.rms_norm(x.view(2, 2, 64), w, x.view(4, 1, 64)),
                lambda: norm.rms_norm_grad(x[:2], x, w), lambda: norm.rms_norm_grad(None, x, w),
                lambda: norm.rms_norm_grad(x, x, w, x[:, :32]), lambda: norm.rms_norm_fp8(x, w)):
        with pytest.raises((ValueError, AttributeError)):
            bad()
    with pytest.raises(RuntimeError, match="derivative"):
        norm.rms_norm_fp8(x, w.clone().requires_grad_())
    l = torch.zeros((4, 8))
    ids = torch.zeros((4, 2), dtype=torch.int32)
    for bad in (lambda: gating.topk_gate(l, 0), lambda: gating.topk_gate(l, 9),
                lambda: gating.topk_gate(l, 2, score="relu"), lambda: gating.topk_gate(l[0], 2),
                lambda: gating.topk_gate(l.double(), 2), lambda: gating.topk_gate(l, 2),
                lambda: gating.topk_gate_grad(l[:, :2], l, ids.long()),
                lambda: gating.topk_gate_grad(l[:, :3], l, ids),
                lambda: gating.topk_gate_grad(l[:, :2], l, ids, score="none")):
        with pytest.raises(ValueError):
            bad()
    codes = torch.zeros((2, 128, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.zeros((2, 1, 1))
    down = torch.zeros((2, 64, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        moe.Fp8MoE(l, (codes, scales), (codes[:1], scales[:1]), 1)
    with pytest.raises(ValueError):
        moe.Fp8MoE(l, (codes, scales), (down, scales), 1, score="none")
    router = torch.zeros((2, 64))
    for layer, rows in ((moe.Fp8MoE(router, (codes, scales), (down, scales), 3), x),
                        (moe.Fp8MoE(router[:1], (codes, scales), (down, scales), 1), x),
                        (moe.Fp8MoE(router.double(), (codes, scales), (down, scales), 1), x),
                        (moe.Fp8MoE(router, (codes, scales), (down, scales), 1), x.float()),
                        (moe.Fp8MoE(router, (codes, scales), (down, scales), 1), x[:, :32]),
                        (moe.Fp8MoE(router, (codes, scales), (down, scales), 1), x)):
        with pytest.raises(ValueError):
            layer.step(rows)
    mlp = moe.Fp8MLP((codes, scales), (down, scales))
    for i, wt in ((ids.long(), l[:, :2]), (ids[:3], l[:3, :2]), (ids, l[:, :3]),
                  (ids, l[:, :2].double())):
        with pytest.raises(ValueError):
            mlp.step_few(x, i, wt)
    # a gradient would be lost
    for layer, rows in ((moe.Fp8MoE(router, (codes, scales), (down, scales), 1), x.clone().requires_grad_()),
                        (moe.Fp8MoE(router.clone().requires_grad_(), (codes, scales), (down, scales), 1), x.cpu())):
        with pytest.raises((RuntimeError, ValueError)):
            layer.step(rows)
    with pytest.raises(RuntimeError):
        mlp.step_few(x.clone().requires_grad_(), ids, l[:, :2])
    q = x.to(torch.float8_e4m3fn)
    for bad in ((x, torch.zeros((1, 4)), codes[0], scales[0]), (q, torch.zeros((4, 1)), codes[0], scales[0]),
                (q, torch.zeros((1, 4)), codes, scales), (q[:, :32], torch.zeros((1, 4)), codes[0], scales[0])):
        with pytest.raises(ValueError):
            fp8.linear_codes(*bad)
    with pytest.raises(ValueError):
        fp8.linear_codes(q, torch.zeros((1, 4)), codes[0], scales[0], torch.float64)


def test_tangents_are_refused():
    x = torch.zeros((4, 64))
    with forward_ad.dual_level():
        d = forward_ad.make_dual(x, torch.ones_like(x))
        for call in (lambda: norm.rms_norm(d, torch.ones(64)), lambda: norm.rms_norm_fp8(d, torch.ones(64)),
                     lambda: norm.rms_norm_grad(d, x, torch.ones(64)), lambda: gating.topk_gate(d, 2),
                     lambda: gating.topk_gate_grad(x[:, :2], d, torch.zeros((4, 2), dtype=torch.int32))):
            with pytest.raises(RuntimeError, match="tangent"):
                call()


# ----------------------------------------------------------- device and stream

OTHER = torch.device("cuda", 1)


class Stream:
    def __init__(self, device):
        self.device = device


class ExternalStream(Stream):
    def __init__(self, handle, device=None):
        super().__init__(device)
        self.handle = handle


class Rows(types.SimpleNamespace):
    """A tensor on the second GPU, as far as the Python side looks at it."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        super().__init__(shape=shape, dtype=dtype, device=OTHER, requires_grad=False)

    def dim(self):
        return len(self.shape)


def moe_layer():
    return moe.Fp8MoE(Rows(4, 64), (Rows(4, 16, 64), Rows(4, 1, 1)), (Rows(4, 64, 8), Rows(4, 1, 1)), 2)


CALLS = [("rms_norm", lambda **s: norm.rms_norm(Rows(4, 64), Rows(64), **s)),
         ("rms_norm_fp8", lambda **s: norm.rms_norm_fp8(Rows(4, 64), Rows(64), **s)),
         ("rms_norm_grad", lambda **s: norm.rms_norm_grad(Rows(4, 64), Rows(4, 64), Rows(64), **s)),
         ("topk_gate", lambda **s: gating.topk_gate(Rows(4, 8), 2, **s)),
         ("topk_gate_grad", lambda **s: gating.topk_gate_grad(Rows(4, 2), Rows(4, 8), Rows(4, 2), **s)),
         ("linear_codes", lambda **s: fp8.linear_codes(Rows(4, 64), Rows(1, 4), Rows(8, 64), Rows(1, 1),
                                                       **s)),
         ("moe_layer", lambda **s: moe_layer().step(Rows(4, 64), **s)),
         ("moe_layer", lambda **s: moe_layer().mlp.step_few(Rows(4, 64), Rows(4, 2), Rows(4, 2), **s))]


@pytest.mark.parametrize("name,call", CALLS)
def test_a_given_stream_is_the_tensors_devices(name, call, monkeypatch):
    now, calls = {"stream": None}, []

    @contextlib.contextmanager
    def on(s):
        before, now["stream"] = now["stream"], s
        yield
        now["stream"] = before

    def record(n):
        def f(*args):
            calls.append((n, now["stream"]))
            return Rows(4, 8), Rows(4, 2), Rows(4, 2)
        return f

    native = types.SimpleNamespace(**{n: record(n) for n, _ in CALLS})
    native.rms_norm = lambda *a: record("rms_norm_fp8" if a[4] else "rms_norm")(*a)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", ExternalStream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    for m in (norm, gating, fp8, tokens):
        monkeypatch.setattr(m, "native", lambda: native)
    monkeypatch.setattr(F, "native", lambda: native)
    call(stream=4242)
    mine = Stream(OTHER)
    call(stream=mine)
    assert [n for n, _ in calls] == [name, name]
    assert calls[0][1].handle == 4242 and calls[0][1].device == OTHER and calls[1][1] is mine
    with pytest.raises(ValueError, match="stream"):
        call(stream=Stream(torch.device("cuda", 0)))
    assert len(calls) == 2
