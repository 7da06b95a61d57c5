"""The binding of the router, the expert layer and the 8-bit calls on the CPU:
what it refuses, and what it keeps, before anything is launched."""
import types

import pytest
import torch

import bit_gemv_q4_b200 as gq

E4M3 = torch.float8_e4m3fn


class OnGpu:
    """What the binding looks at of a tensor on one of several GPUs; its memory is never touched."""

    def __init__(self, *shape, dtype=torch.float32, gpu=0):
        self.shape, self.dtype, self.gpu = torch.Size(shape), dtype, gpu
        self.device = types.SimpleNamespace(type="cuda", index=gpu)

    is_cuda = True

    def get_device(self):
        return self.gpu

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000000


@pytest.fixture
def two_gpus(monkeypatch):
    """Two GPUs, of which 0 is the current one, and a library that must not be reached."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0)

    def launched(*args):
        raise AssertionError("launched")
    for name in ("gq_moe_route", "gq_moe_q4_0_tiled", "gq_moe_ksb_tiled", "gq_quantize_fp8", "gq_dequantize_fp8",
                 "gq_gemm_fp8"):
        monkeypatch.setattr(gq.lib, name, launched)


def calls():
    """(call, its tensors by name) of every entry point, all of them given."""
    u8, i32, f16 = torch.uint8, torch.int32, torch.float16
    st = OnGpu(1, dtype=i32)
    ws = OnGpu(1 << 20, dtype=u8)
    route = dict(x=OnGpu(4, 64), Wr=OnGpu(8, 64), bias=OnGpu(8), ids=OnGpu(4, 2, dtype=i32), weights=OnGpu(4, 2),
                 workspace=ws, dev_status=st)
    yield lambda **t: gq.gq_moe_route(k=2, flags=gq.GQ_ROUTE_SIGMOID, **t), route
    for call, n in ((gq.gq_moe_q4_0_tiled, 64), (gq.gq_moe_ksb_tiled, 256)):
        layer = dict(gate=OnGpu(1 << 20, dtype=u8), up=OnGpu(1 << 20, dtype=u8), down=OnGpu(1 << 20, dtype=u8),
                     x=OnGpu(3, n, dtype=f16), ids=OnGpu(3, 2, dtype=i32), weights=OnGpu(3, 2),
                     out=OnGpu(3, n, dtype=f16), workspace=ws, dev_status=st)
        yield lambda call=call, n=n, **t: call(E=4, I=n, **t), layer
    q, s = OnGpu(4, 256, dtype=E4M3), OnGpu(4, 2)
    yield lambda **t: gq.gq_quantize_fp8(rows=1, **t), dict(x=OnGpu(4, 256), out=q, scales=s, dev_status=st)
    yield lambda **t: gq.gq_dequantize_fp8(rows=1, **t), dict(q=q, scales=s, out=OnGpu(4, 256))
    yield gq.gq_gemm_fp8, dict(W=OnGpu(300, 256, dtype=E4M3), w_scales=OnGpu(3, 2), X=q, x_scales=s,
                               out=OnGpu(4, 300), workspace=ws, dev_status=st)


def test_tensors_of_two_gpus_in_one_call_are_refused(two_gpus):
    for call, tensors in calls():
        with pytest.raises(AssertionError, match="launched"):
            call(**tensors)
        first = next(iter(tensors))
        for name in tensors:
            if name == first:  # (it sets the device; the next one is then elsewhere)
                continue
            other = OnGpu(*tensors[name].shape, dtype=tensors[name].dtype, gpu=1)
            with pytest.raises(ValueError, match="one CUDA device"):
                call(**dict(tensors, **{name: other}))


def test_tensors_on_the_host_are_refused(two_gpus):
    for call, tensors in calls():
        for name in tensors:
            host = torch.zeros(tensors[name].shape).to(tensors[name].dtype)
            with pytest.raises(ValueError, match="CUDA device"):
                call(**dict(tensors, **{name: host}))


def codes(R, K):
    return torch.zeros(R, K).to(torch.float8_e4m3fn)


def test_scales_of_another_block_shape_are_refused():
    W, X = codes(256, 512), codes(4, 512)
    right, xs = torch.zeros(2, 4), torch.zeros(4, 4)
    for bad in (torch.zeros(256, 4),        # scales of 1 x 128 blocks
                torch.zeros(2, 5),          # rows further apart
                torch.zeros(4, 2), torch.zeros(3, 4), torch.zeros(9), torch.zeros(2, 4).double()):
        with pytest.raises(ValueError, match="scale"):
            gq.gq_gemm_fp8(W, bad, X, xs)
        with pytest.raises(ValueError, match="scale"):
            gq.gq_dequantize_fp8(W, bad, 128)
        with pytest.raises(ValueError, match="scale"):
            gq.gq_quantize_fp8(torch.zeros(256, 512), 128, out=W, scales=bad)
    for bad in (torch.zeros(1, 4), torch.zeros(5, 4), torch.zeros(2, 8), torch.zeros(4, 5)):
        with pytest.raises(ValueError, match="scale"):
            gq.gq_gemm_fp8(W, right, X, bad)
    gq._fp8_pair(W, right, 128, "W")            # as they are made
    gq._fp8_pair(W, right.view(-1), 128, "W")   # or in one row


def test_workspace_sizes_are_each_gpus_own(monkeypatch):
    # two GPUs with other numbers of SMs, on which the same product is cut into other pieces
    current = [0]
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0)
    monkeypatch.setattr(gq.lib, "gq_gemm_fp8_workspace_bytes", lambda M, K, B: 1000 * (current[0] + 1))
    monkeypatch.setattr(gq.lib, "gq_gemm_fp8", lambda *args: 0)
    asked = []
    monkeypatch.setattr(gq, "_auto_workspace", lambda name, need, device, stream: asked.append(need) or (None, None, need))
    for gpu in (0, 1, 0, 1):
        current[0] = gpu
        gq.gq_gemm_fp8(OnGpu(301, 272, dtype=E4M3, gpu=gpu), OnGpu(3, 3, gpu=gpu), OnGpu(41, 272, dtype=E4M3, gpu=gpu),
                       OnGpu(41, 3, gpu=gpu), out=OnGpu(41, 301, gpu=gpu))
    assert asked == [1000, 2000, 1000, 2000]
