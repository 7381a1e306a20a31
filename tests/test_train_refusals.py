"""Refusals of the training calls and of the dense product with a fused epilogue: host checks
(CPU) and the argument errors that need a device (gpu)."""
import ctypes as C

import pytest
import torch

from routing_dispatch_grouped_top_b200 import binding as B
from routing_dispatch_grouped_top_b200 import build

OK, INVALID, UNSUPPORTED, WORKSPACE, NO_DEVICE = 0, 1, 2, 3, 7
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


@pytest.mark.parametrize("M,N,Kd,code", [(-1, 64, 64, INVALID), (4, 0, 64, INVALID), (4, 64, 7, INVALID),
                                         (4, 12, 64, UNSUPPORTED), (4, 64, 20, UNSUPPORTED),
                                         (1 << 31, 64, 64, UNSUPPORTED)])
def test_dense_shapes(lib, M, N, Kd, code):
    assert lib.moe_dense_workspace_bytes(M, N, Kd) == 0
    assert lib.moe_dense_epilogue(None, None, None, None, 0, M, N, Kd, None, None, None, 0, None) == code
    assert lib.moe_dense_backward(None, None, None, None, 0, M, N, Kd, None, None, None, None, 0, None, 0, None) == code


def test_dense_activation_and_gradient_flags(lib):
    for act in (-1, 5):
        assert lib.moe_dense_epilogue(None, None, None, None, act, 4, 64, 64, None, None, None, 0, None) == INVALID
        assert lib.moe_dense_backward(None, None, None, None, act, 4, 64, 64, None, None, None, None, 0, None, 0,
                                      None) == INVALID
    for flags in (2, 4, 7):   # accumulating needs fp32 gradients; unknown flags
        assert lib.moe_dense_backward(None, None, None, None, 0, 4, 64, 64, None, None, None, None, flags, None, 0,
                                      None) == INVALID
    n = lib.moe_dense_workspace_bytes(4, 64, 64)
    assert n >= 256 and n % 256 == 0


def test_layer_shapes(lib):
    for d, code in ((B.dims(T=4, H=60, E=8, K=2, F=64), UNSUPPORTED), (B.dims(T=4, H=64, E=8, K=9, F=64), INVALID),
                    (B.dims(T=1 << 30, H=64, E=64, K=8, F=64), UNSUPPORTED)):
        r = C.byref(d)
        assert lib.moe_grouped_gate_up_train(None, None, None, None, r, None, None, None, None, 0, None) == code
        assert lib.moe_grouped_ffn_backward(*[None] * 9, r, *[None] * 6, 0, None, 0, None) == code
        assert lib.moe_combine_backward(None, None, None, None, r, None, None, None) == code


def test_binding_checks_types_and_shapes(lib):
    a, w, out = torch.zeros((4, 64), dtype=BF), torch.zeros((8, 64), dtype=BF), torch.zeros((4, 8), dtype=BF)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.moe_dense_epilogue(a, w, out, ws)
    with pytest.raises(ValueError, match="float32 gradients"):
        B._grad_flags(True, dw=torch.zeros(1, dtype=BF))
    with pytest.raises(ValueError, match="all torch.float32 or all torch.bfloat16"):
        B._grad_flags(False, dw_gate=torch.zeros(1, dtype=BF), dw_up=torch.zeros(1))
    with pytest.raises(ValueError, match="all torch.float32"):
        B._grad_flags(False, dw=torch.zeros(1, dtype=torch.float16))
    with pytest.raises(ValueError, match="act must be"):
        B._act("swish")
    with pytest.raises(ValueError, match="invalid dense shape"):
        B.make_dense_workspace(4, 12, 64)


@pytest.mark.gpu
def test_null_misaligned_and_short_arguments(lib, cuda_ok):
    dev = "cuda"
    a, w, out = (torch.zeros(s, dtype=BF, device=dev) for s in ((4, 64), (8, 64), (4, 8)))
    ws = B.make_dense_workspace(4, 8, 64)
    args = [a.data_ptr(), w.data_ptr(), None, None, 0, 4, 8, 64, out.data_ptr(), None, ws.data_ptr(), ws.numel(), None]
    for i in (0, 1, 8):
        bad = list(args)
        bad[i] = None
        assert lib.moe_dense_epilogue(*bad) == INVALID
        bad[i] = args[i] + 2   # bf16 rows start on 16-byte boundaries
        assert lib.moe_dense_epilogue(*bad) == INVALID
    for ptr, n in ((None, 256), (ws.data_ptr(), 255), (ws.data_ptr() + 16, 256)):
        bad = list(args)
        bad[10], bad[11] = ptr, n
        assert lib.moe_dense_epilogue(*bad) == WORKSPACE
    with pytest.raises(ValueError, match="out has shape"):
        B.moe_dense_epilogue(a, w, torch.zeros((4, 16), dtype=BF, device=dev), ws)
    with pytest.raises(ValueError, match="residual has shape"):
        B.moe_dense_epilogue(a, w, out, ws, residual=torch.zeros((8, 4), dtype=BF, device=dev))
    with pytest.raises(ValueError, match="dw has shape"):
        B.moe_dense_backward(out, a, w, None, None, None, torch.zeros((64, 8), dtype=BF, device=dev), None, ws)
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.moe_dense_epilogue(a, w, out, ws, bias=torch.zeros(8))
    # an activation needs the pre-activations, and a place for dpre where a product follows
    pre = torch.zeros((4, 8), device=dev)
    da = torch.zeros((4, 64), dtype=BF, device=dev)
    with pytest.raises(B.MoEError):
        B.moe_dense_backward(out, a, w, None, out.clone(), da, None, None, ws, act="silu")
    with pytest.raises(B.MoEError):
        B.moe_dense_backward(out, a, w, pre, None, da, None, None, ws, act="silu")
    with pytest.raises(B.MoEError):
        B.moe_dense_backward(out, a, None, None, None, da, None, None, ws)
    with pytest.raises(ValueError, match="contiguous"):
        B.moe_dense_epilogue(torch.zeros((64, 4), dtype=BF, device=dev).t(), w, out, ws)
    d = B.dims(T=4, H=64, E=2, K=1, F=16)
    lws = B.make_workspace(d)
    x, off = torch.zeros((4, 64), dtype=BF, device=dev), torch.tensor([0, 2, 4], dtype=torch.int32, device=dev)
    gw, dw = torch.zeros((2, 16, 64), dtype=BF, device=dev), torch.zeros((2, 64, 16), dtype=BF, device=dev)
    f, h = torch.zeros((4, 16), device=dev), torch.zeros((4, 16), dtype=BF, device=dev)
    with pytest.raises(B.MoEError):   # dw_gate without dw_up
        B.moe_grouped_ffn_backward(x, f, f, h, x, off, gw, gw, dw, d, h, h, None, gw, None, None, lws)
    with pytest.raises(B.MoEError):   # dxp without dg
        B.moe_grouped_ffn_backward(x, f, f, h, x, off, gw, gw, dw, d, None, h, x, None, None, None, lws)
    with pytest.raises(ValueError, match="holds"):
        B.moe_grouped_gate_up_train(x[:3].contiguous(), off, gw, gw, d, f, f, h, lws)
    with pytest.raises(ValueError, match="must be torch.float32"):
        B.moe_grouped_gate_up_train(x, off, gw, gw, d, h, h, h, lws)
    with pytest.raises(B.MoEError):   # dw without y
        B.moe_combine_backward(x, None, torch.zeros(4, dtype=torch.int32, device=dev), f[:, :1].contiguous(), d, None,
                               f[:, :1].contiguous())
    assert B.read_device_status(lws) == 0


def test_extents_that_round_up_past_32_bits(lib):
    top = (1 << 31) - 8
    for M, N, Kd in ((top, 8, 8), (4, top, 8), (4, 8, top)):
        assert lib.moe_dense_workspace_bytes(M, N, Kd) == 0
        assert lib.moe_dense_epilogue(None, None, None, None, 0, M, N, Kd, None, None, None, 0, None) == UNSUPPORTED
        assert lib.moe_dense_backward(None, None, None, None, 0, M, N, Kd, None, None, None, None, 0, None, 0,
                                      None) == UNSUPPORTED
    assert lib.moe_dense_workspace_bytes((1 << 31) - 1032, 8, 8) > 0


@pytest.mark.gpu
def test_rows_that_round_up_past_32_bits(lib, cuda_ok):
    r = C.byref(B.dims(T=(1 << 31) - 8, H=64, E=2, K=1, F=64))
    assert lib.moe_grouped_gate_up_train(None, None, None, None, r, None, None, None, None, 0, None) == UNSUPPORTED
    assert lib.moe_grouped_ffn_backward(*[None] * 9, r, *[None] * 6, 0, None, 0, None) == UNSUPPORTED


@pytest.mark.parametrize("H,F", [((1 << 31) - 8, 8), (8, (1 << 31) - 8), ((1 << 31) - 1024, 8), (8, (1 << 31) - 1024)])
def test_layer_widths_that_round_up_past_32_bits(lib, H, F):
    r = C.byref(B.dims(T=4, H=H, E=1, K=1, F=F))
    assert lib.moe_grouped_gate_up_train(None, None, None, None, r, None, None, None, None, 0, None) == UNSUPPORTED
    assert lib.moe_grouped_ffn_backward(*[None] * 9, r, *[None] * 6, 0, None, 0, None) == UNSUPPORTED


def test_widest_layer_is_not_refused_for_its_width(lib):
    top = (1 << 31) - 1032   # refused for what comes next: no device, or no workspace
    for H, F in ((top, 8), (8, top)):
        r = C.byref(B.dims(T=4, H=H, E=1, K=1, F=F))
        code = lib.moe_grouped_gate_up_train(None, None, None, None, r, None, None, None, None, 0, None)
        assert code == (WORKSPACE if torch.cuda.is_available() else NO_DEVICE)
