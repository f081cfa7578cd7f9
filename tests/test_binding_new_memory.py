"""Where the helpers' outputs come from: torch's short way when it behaves as they need, its public one
otherwise.  On the CPU, with stand-ins for the short way."""
import pytest

from tiled_online_softmax_sm_gb300 import binding as fb

torch = pytest.importorskip("torch")


def _cpu(size, strides, dtype):
    return torch.empty_strided(size, strides, dtype=dtype)


STAND_INS = {
    "another signature": lambda size, strides, dtype, device: _cpu(size, strides, dtype),
    "raises": lambda size, strides, dtype: (_ for _ in ()).throw(RuntimeError("no")),
    "another type": lambda size, strides, dtype: _cpu(size, strides, torch.int64),
    "another layout": lambda size, strides, dtype: torch.empty(size, dtype=dtype),
    "another device": _cpu,
    "no tensor": lambda size, strides, dtype: None,
}


@pytest.mark.parametrize("short", [None, *STAND_INS.values()], ids=["missing", *STAND_INS])
def test_short_way_that_does_not_fit_is_passed_over(short, monkeypatch):
    for name in ("_current_raw_stream", "_current_device", "_CODES", "_SCALES", "_I32", "_BF16", "_F32", "_U8", "_new"):
        monkeypatch.setattr(fb, name, None)
    guards = torch._C._dynamo.guards
    if short is None:
        monkeypatch.delattr(guards, "_empty_strided_cuda", raising=False)
    else:
        monkeypatch.setattr(guards, "_empty_strided_cuda", short, raising=False)
    fb._bind_torch()
    assert fb._new is fb._new_strided


def test_short_way_that_fits_is_taken(monkeypatch):
    monkeypatch.setattr(fb, "_new", None)
    assert fb._fits(_cpu, "cpu") and not fb._fits(_cpu, "cuda")
