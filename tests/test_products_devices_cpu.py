"""Calls on a given stream of the products grouped by expert and the microscaled operators: operands and streams
of another device than the current one are refused.  Without a GPU: a stand-in for the library notes its calls,
CPU tensors that name a GPU stand for device ones."""
import types

import pytest
import torch

from mixture_experts_ffn_gemm_gb300 import binding as B
from test_products_cpu import OnAnother, OnDevice

BF16, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
R, E, N, K = 10, 3, 16, 64


@pytest.fixture
def calls(moelib, monkeypatch):
    """Calls that reach the library, which is taken for the real one; the current device is 0."""
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append(name) or B.MOE_OK

    lib = Library()
    monkeypatch.setattr(B, "_lib", lib)
    monkeypatch.setattr(B, "_address", lambda name: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    return made


def _calls_of(kind, stream):
    z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype).as_subclass(kind)  # noqa: E731
    offs, ws, f = z(E + 1, dtype=I32), z(256, dtype=U8), z(1, dtype=F32)
    codes, scales = z(R, K // 2, dtype=U8), z(B._scale_bytes(R, K, E, 1), dtype=U8)
    w, ws_ = z(E * N, K // 2, dtype=U8), z(B._scale_bytes(E * N, K, E, 1), dtype=U8)
    q = B.make_micro_config(R, K, "nv", groups=E)
    return [
        lambda: B.moe_grouped_product(B.make_product_config(R, E, N, K), offs, z(R, K), z(E, N, K), z(R, N), ws,
                                      stream=stream),
        lambda: B.moe_micro_quantize(q, z(R, K), None, offs, f, codes, scales, ws, stream=stream),
        lambda: B.moe_micro_dequantize(q, codes, scales, offs, f, z(R, K), ws, stream=stream),
        lambda: B.moe_micro_product(B.make_micro_product_config(R, E, N, K, "nv"), offs, codes, scales, f, w, ws_,
                                    None, z(R, N), ws, stream=stream)]


def _stream(device, handle):
    return types.SimpleNamespace(device=torch.device("cuda", device), cuda_stream=handle)


@pytest.mark.parametrize("stream", [0, 0x1234, _stream(1, 0), _stream(1, 0x1234), _stream(0, 0x1234)])
def test_operands_of_another_device_are_refused(calls, stream):
    for call in _calls_of(OnAnother, stream):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert calls == []


@pytest.mark.parametrize("handle", [0, 0x1234])
def test_streams_of_another_device_are_refused(calls, handle):
    for call in _calls_of(OnDevice, _stream(1, handle)):
        with pytest.raises(ValueError, match="stream: of device 1"):
            call()
    assert calls == []


@pytest.mark.parametrize("stream", [0, 0x1234, _stream(0, 0x1234)])
def test_operands_and_streams_of_the_current_device_are_taken(calls, stream):
    for call in _calls_of(OnDevice, stream):
        call()
    assert calls == ["moe_grouped_product", "moe_micro_quantize", "moe_micro_dequantize", "moe_micro_product"]


def test_another_current_device(calls, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for call in _calls_of(OnAnother, _stream(1, 0)):
        call()
    assert len(calls) == 4
    for call in _calls_of(OnDevice, 0):
        with pytest.raises(ValueError, match="current device is 1"):
            call()


def test_operands_outside_any_gpu_are_refused_before_a_device_is_asked_for(calls, monkeypatch):
    def none():
        raise RuntimeError("no driver")

    monkeypatch.setattr(torch._C, "_cuda_getDevice", none)
    for call in _calls_of(torch.Tensor, 0):
        with pytest.raises(ValueError, match="ws"):
            call()
    assert calls == []
