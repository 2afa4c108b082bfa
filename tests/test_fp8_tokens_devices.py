"""Which device and stream a call of the token and FP8 operators runs on, when its
tensors lie on another GPU than the current one.  No GPU: torch's contexts and the
library's entry points are stand-ins that record what is current when they are
called."""
import contextlib
import types

import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import fp8, moe, tokens
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F

OTHER = torch.device("cuda", 1)


class Stream:
    def __init__(self, device):
        self.device = device


class ExternalStream(Stream):
    def __init__(self, handle, device=None):
        super().__init__(torch.device("cuda", 0) if device is None else device)
        self.handle = handle


class Rows(types.SimpleNamespace):
    """A tensor on the second GPU, as far as the Python side looks at it."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        super().__init__(shape=shape, dtype=dtype, device=OTHER, requires_grad=False)

    def dim(self):
        return len(self.shape)

    def stride(self, i):
        return self.shape[1] if i == 0 else 1

    def data_ptr(self):
        return 0

    def contiguous(self):
        return self

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape[0] * self.shape[1]

    def view(self, *shape):
        return self

    def __getitem__(self, i):
        return self


@pytest.fixture
def seen(monkeypatch):
    """Calls of the library as (name, current device, current stream or None)."""
    now = {"device": 0, "stream": None}
    calls = []

    @contextlib.contextmanager
    def on(device, stream=None):
        before = dict(now)
        now.update(device=device.index, stream=stream)
        yield
        now.update(before)

    def record(name, result=None):
        def call(*args, **kw):
            calls.append((name, now["device"], now["stream"]))
            return result
        return call

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", ExternalStream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: on(s.device, s))
    monkeypatch.setattr(torch.cuda, "device_of", lambda t: on(t.device, now["stream"]))
    native = types.SimpleNamespace(**{n: record(n, Rows(4, 8)) for n in (
        "dispatch", "combine", "combine_grad", "linear", "expert_linear")})
    monkeypatch.setattr(tokens, "native", lambda: native)
    monkeypatch.setattr(fp8, "native", lambda: native)
    monkeypatch.setattr(F, "nvfp4_fp8_quantize", record("quantize"))
    monkeypatch.setattr(F, "nvfp4_fp8_quantize_weights", record("quantize_weights"))
    monkeypatch.setattr(F, "moe_route", record("route", (Rows(5), None, None, Rows(8))))
    monkeypatch.setattr(torch, "empty", lambda shape, **kw: Rows(*shape))
    return calls


def layer():
    return moe.Fp8MLP((Rows(4, 16, 64), Rows(4, 1, 1)), (Rows(4, 64, 8), Rows(4, 1, 1)))


CALLS = [("dispatch", lambda **s: tokens.dispatch(Rows(4, 64), Rows(4, 2), **s)),
         ("dispatch_grad", lambda **s: tokens.dispatch_grad(Rows(8, 64), Rows(4, 2), **s)),
         ("combine", lambda **s: tokens.combine(Rows(8, 64), Rows(4, 2), **s)),
         ("combine_grad", lambda **s: tokens.combine_grad(Rows(4, 64), Rows(8, 64), Rows(4, 2),
                                                          Rows(4, 2), **s)),
         ("linear", lambda **s: fp8.linear(Rows(4, 64), Rows(8, 64), Rows(1, 1), **s)),
         ("expert_linear", lambda **s: fp8.expert_linear(Rows(4, 64), Rows(4, 8, 64),
                                                         Rows(4, 1, 1), Rows(5), **s)),
         ("quantize_rows", lambda **s: fp8.quantize_rows(Rows(4, 64), **s)),
         ("quantize_weights", lambda **s: fp8.quantize_weights(Rows(4, 8, 64), **s)),
         ("Fp8MLP.route", lambda **s: layer().route(Rows(4, 2, dtype=torch.int32), **s)),
         ("Fp8MLP.step", lambda **s: layer().step(Rows(4, 64), Rows(4, 2, dtype=torch.int32),
                                                  Rows(4, 2, dtype=torch.float32), **s))]


@pytest.mark.parametrize("name,call", CALLS, ids=[c[0] for c in CALLS])
def test_a_given_stream_is_the_tensors_devices(name, call, seen):
    call(stream=4242)
    assert seen
    for _, device, stream in seen:
        assert device == 1 and stream.handle == 4242 and stream.device == OTHER
    del seen[:]
    mine = Stream(OTHER)
    call(stream=mine)
    assert seen and all(device == 1 and stream is mine for _, device, stream in seen)
    del seen[:]
    with pytest.raises(ValueError, match="stream"):
        call(stream=Stream(torch.device("cuda", 0)))
    assert not seen


@pytest.mark.parametrize("call", [c[1] for c in CALLS if c[0] in (
    "quantize_rows", "quantize_weights", "Fp8MLP.route")])
def test_calls_without_a_guard_of_their_own_switch_the_device(call, seen):
    call()
    assert seen and all(device == 1 for _, device, _ in seen)


def test_step_routes_on_the_tensors_device(seen):
    layer().step(Rows(4, 64), Rows(4, 2, dtype=torch.int32), Rows(4, 2, dtype=torch.float32))
    assert ("route", 1, None) in seen


def test_operands_of_the_quantiser_share_a_device(seen):
    pos = Rows(4, 2, dtype=torch.int32)
    pos.device = torch.device("cuda", 0)
    with pytest.raises(ValueError, match="devices"):
        fp8.quantize_rows(Rows(4, 64), pos)
    assert not seen


def test_cpu_tensors_with_a_stream_are_refused():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fp8.quantize_rows(x, stream=1)
    with pytest.raises(ValueError):
        tokens.dispatch(x, torch.zeros((4, 2), dtype=torch.int32), stream=1)
