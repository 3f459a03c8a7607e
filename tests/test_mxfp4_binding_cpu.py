"""What the binding of the MXFP4 and gated calls refuses before the library is called: workspaces and
tensors that the library cannot see to be wrong.  With stand-ins for tensors on CUDA devices."""
import importlib.util
import sys

import pytest
import torch

import sparse_expert_ffn_route_gb300 as moe
from sparse_expert_ffn_route_gb300 import binding


class OnDevice:
    """As much of a tensor on a CUDA device as the binding looks at."""

    def __init__(self, *shape, dtype=torch.bfloat16, device=0, contiguous=True):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, "cuda:%d" % device if device >= 0 else "cpu"
        self._device, self._contiguous = device, contiguous

    def get_device(self):
        return self._device

    @property
    def is_cuda(self):
        return self._device >= 0

    def is_contiguous(self):
        return self._contiguous

    def stride(self, i):
        return (2 * self.shape[1], 1)[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 1 << 20


class NoStream:
    cuda_stream = 0


class Called(Exception):
    pass


class Library:
    def __getattr__(self, name):
        def call(*a):
            raise Called(name)
        return call


@pytest.fixture
def bound(monkeypatch):
    """The binding over a library that only says that it was called; the current device of two is 0."""
    monkeypatch.setattr(binding, "load_library", lambda: Library())
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_device_count", lambda: 2)


def calls():
    """name -> (function of keyword tensors, its tensors)"""
    u8, i32 = torch.uint8, torch.int32
    cfg = moe.MoeConfig.make(128, 2, 1, 64)
    w = {"w_gate": OnDevice(2, 64, 64, dtype=u8), "s_gate": OnDevice(2, 64, 4, dtype=u8), "w_up": OnDevice(2, 64, 64, dtype=u8),
         "s_up": OnDevice(2, 64, 4, dtype=u8), "w_down": OnDevice(2, 128, 32, dtype=u8), "s_down": OnDevice(2, 128, 2, dtype=u8)}
    ws, s = OnDevice(4096, dtype=u8), NoStream
    return {
        "quantize": (lambda **t: moe.moe_quantize_mxfp4(**t, stream=s),
                     dict(x=OnDevice(4, 64), codes=OnDevice(4, 32, dtype=u8), scales=OnDevice(4, 2, dtype=u8))),
        "dequantize": (lambda **t: moe.moe_dequantize_mxfp4(**t, stream=s),
                       dict(codes=OnDevice(4, 32, dtype=u8), scales=OnDevice(4, 2, dtype=u8), y=OnDevice(4, 64))),
        "matmul": (lambda **t: moe.moe_mxfp4_matmul(**t, stream=s),
                   dict(x=OnDevice(4, 32, dtype=u8), x_scales=OnDevice(4, 2, dtype=u8), w=OnDevice(8, 32, dtype=u8),
                        w_scales=OnDevice(8, 2, dtype=u8), y=OnDevice(4, 8), workspace=ws, offsets=OnDevice(2, dtype=i32))),
        "experts": (lambda **t: moe.moe_mxfp4_expert_ffn(cfg, weights=w, **t, stream=s),
                    dict(x=OnDevice(4, 128), y_pairs=OnDevice(4, 128), workspace=ws, offsets=OnDevice(3, dtype=i32),
                         tok=OnDevice(4, dtype=i32))),
        "forward": (lambda **t: moe.moe_gated_forward(**t, stream=s),
                    dict(x=OnDevice(4, 64), w_gate=OnDevice(32, 64), w_up=OnDevice(32, 64), h=OnDevice(4, 32), workspace=ws,
                         g=OnDevice(4, 32), u=OnDevice(4, 32))),
        "backward": (lambda **t: moe.moe_gated_backward(**t, stream=s),
                     dict(dh=OnDevice(4, 32), x=OnDevice(4, 64), w_gate=OnDevice(32, 64), w_up=OnDevice(32, 64), g=OnDevice(4, 32),
                          u=OnDevice(4, 32), dx=OnDevice(4, 64), dw_gate=OnDevice(32, 64), dw_up=OnDevice(32, 64), workspace=ws)),
    }


NAMES = ("quantize", "dequantize", "matmul", "experts", "forward", "backward")


@pytest.mark.parametrize("name", NAMES)
def test_right_tensors_reach_the_library(bound, name):
    call, tensors = calls()[name]
    with pytest.raises(Called):
        call(**tensors)


@pytest.mark.parametrize("name", NAMES[2:])
@pytest.mark.parametrize("bad", [dict(device=-1), dict(device=1), dict(contiguous=False), dict(dtype=torch.float32)])
def test_workspace_is_bytes_on_the_same_device(bound, name, bad):
    call, tensors = calls()[name]
    with pytest.raises(ValueError, match="workspace"):
        call(**{**tensors, "workspace": OnDevice(4096, **{"dtype": torch.uint8, **bad})})


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("device", [-1, 1])
def test_every_tensor_is_on_the_same_device(bound, name, device):
    call, tensors = calls()[name]
    for k, t in tensors.items():
        with pytest.raises(ValueError):
            call(**{**tensors, k: OnDevice(*t.shape, dtype=t.dtype, device=device)})


@pytest.mark.parametrize("name", NAMES)
def test_the_device_is_the_current_one(bound, monkeypatch, name):
    monkeypatch.setattr(binding, "_current_device", lambda: 1)
    call, tensors = calls()[name]
    with pytest.raises(ValueError, match="current device"):
        call(**tensors)


def test_import_without_torchs_private_stream_call(monkeypatch):
    """The binding imports on a torch that lacks it, and asks for the stream the public way."""
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    spec = importlib.util.spec_from_file_location("binding_without", binding.__file__)
    copy = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, spec.name, copy)
    spec.loader.exec_module(copy)
    asked = []

    class Stream:
        cuda_stream = 77
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: asked.append(device) or Stream)
    assert copy._raw_stream(None, 3) == 77 and asked == [3]
