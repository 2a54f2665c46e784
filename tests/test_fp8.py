"""Refusals of the 8-bit entry points, on the host before anything is enqueued."""
import ctypes

import pytest
import torch

import fp8_ref as ref
from sparse_mixture_experts_amd import moe

A = 1 << 20  # a fake, 16-byte aligned device address; never dereferenced here


@pytest.fixture(scope="module")
def lib():
    return moe.load()


@pytest.mark.parametrize("args", [
    (-1, 4, 16, A, 1, 1, A, A), (1, -4, 16, A, 1, 1, A, A), (1, 4, 0, A, 1, 1, A, A), (1, 4, 24, A, 1, 1, A, A),
    (1, 4, 16, A, 3, 1, A, A), (1, 4, 16, A, 1, 64, A, A), (1, 4, 16, None, 1, 1, A, A), (1, 4, 16, A + 8, 1, 1, A, A),
    (1, 4, 16, A, 1, 1, None, A), (1, 4, 16, A, 1, 1, A, None), (1, 4, 16, A, 1, 1, A + 4, A),
    (1 << 20, 1 << 20, 16, A, 1, 1, A, A),       # more rows than an int32 counts
    (1 << 15, 1 << 10, 16 << 10, A, 1, 128, A, A),  # more workgroups than a grid holds
    (1, (1 << 31) - 1, 16, A, 1, 128, A, A), (1, 1, (1 << 31) - 16, A, 1, 128, A, A),  # sizes that a rounding up overflows
    (1, 1, (1 << 31) - 16, A, 1, 1, A, A), (1 << 30, 1 << 30, (1 << 31) - 16, A, 1, 1, A, A),
])
def test_quantize_refusals(lib, args):
    assert lib.moe_fp8_quantize(*args, None) == moe.MOE_E_INVALID


def test_quantize_of_nothing(lib):
    assert lib.moe_fp8_quantize(0, 4, 16, A, 1, 1, A, A, None) == moe.MOE_OK
    assert lib.moe_fp8_quantize(4, 0, 16, A, 1, 128, A, A, None) == moe.MOE_OK


GOOD = dict(rows=4, N=32, K=64, n_experts=2, a_rows=4, a=A, a_scales=A, row_map=A, expert_off=A, w=A, w_scales=A, y=A,
            out_dtype=1)


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(N=0), dict(N=24), dict(K=0), dict(K=40), dict(N=1 << 16, K=(1 << 15) + 16),
    dict(n_experts=0), dict(n_experts=1025), dict(a_rows=-1), dict(a_rows=0), dict(a_rows=3, row_map=None),
    dict(out_dtype=3), dict(a=None), dict(a_scales=None), dict(w=None), dict(w_scales=None), dict(y=None),
    dict(expert_off=None), dict(a=A + 1), dict(row_map=A + 4), dict(y=A + 8), dict(expert_off=A + 4),
    dict(rows=1 << 30, N=1 << 14, n_experts=1),  # more workgroups than a grid holds
])
def test_product_refusals(lib, change):
    assert lib.moe_fp8_matmul(*{**GOOD, **change}.values(), None) == moe.MOE_E_INVALID


def test_product_of_nothing(lib):
    assert lib.moe_fp8_matmul(*{**GOOD, "rows": 0}.values(), None) == moe.MOE_OK
    assert lib.moe_fp8_matmul(*{**GOOD, "rows": 0, "a_rows": 0, "n_experts": 1, "expert_off": None,
                                "row_map": None}.values(), None) == moe.MOE_OK


@pytest.mark.parametrize("args", [
    (-1, 16, 16, A, A, A, A), (1, 8, 16, A, A, A, A), (1, 16, 0, A, A, A, A), (1, 16, 16, None, A, A, A),
    (1, 16, 16, A, A, A + 4, A), (1 << 24, 16, 16, A, A, A, A),
    (1, (1 << 31) - 16, 16, A, A, A, A), (1, 16, (1 << 31) - 16, A, A, A, A),
    ((1 << 31) - 1, (1 << 31) - 16, (1 << 31) - 16, A, A, A, A),
])
def test_transpose_refusals(lib, args):
    assert lib.moe_fp8_transpose(*args, None) == moe.MOE_E_INVALID


def test_transpose_of_nothing(lib):
    assert lib.moe_fp8_transpose(0, 16, 16, None, None, None, None, None) == moe.MOE_OK


def test_layer_refusals(lib):
    size = ctypes.c_size_t()
    for act in ("f32", "bf16", "f16"):
        d = moe.make_desc(272, 144, 8, 2, act=act, wfmt="fp8")
        assert lib.moe_workspace_size(ctypes.byref(d), 4, ctypes.byref(size)) == moe.MOE_OK
    for D, F in ((264, 144), (272, 136)):
        d = moe.make_desc(D, F, 8, 2, wfmt="fp8")
        assert lib.moe_workspace_size(ctypes.byref(d), 4, ctypes.byref(size)) == moe.MOE_E_INVALID
    d = moe.make_desc(272, 144, 8, 2, wfmt="fp8")
    need = moe.moe_workspace_size(d, 0)
    none = moe.Proj(None, None, None)

    def forward(p):
        w = moe.Weights(A, None, p, moe.Proj(A, A, None), none, moe.Proj(A, A, None))
        return lib.moe_forward(ctypes.byref(d), 0, A, ctypes.byref(w), A, 1, None, None, A, need, None)

    assert forward(moe.Proj(A, A, None)) == moe.MOE_OK
    assert forward(moe.Proj(A, None, None)) == moe.MOE_E_INVALID     # scales missing
    assert forward(moe.Proj(A, A, A)) == moe.MOE_E_INVALID           # no biases in this format
    assert forward(moe.Proj(A, A, None, A)) == moe.MOE_E_INVALID     # nor a tile-packed copy
    assert forward(moe.Proj(A, A + 4, None)) == moe.MOE_E_INVALID
    assert lib.moe_packed_bytes(ctypes.byref(d), moe.MOE_PROJ_DOWN, ctypes.byref(size)) == moe.MOE_E_UNSUPPORTED


@pytest.mark.parametrize("shape", [
    dict(d_model=2048, d_ff=768, n_experts=128, top_k=8), dict(d_model=272, d_ff=144, n_experts=4, top_k=2, n_shared=2),
])
def test_workspace_covers_smaller_T(shape):
    d, prev = moe.make_desc(wfmt="fp8", **shape), 0
    for T in range(0, 2200, 7):
        size = moe.moe_workspace_size(d, T)
        assert size >= prev
        prev = size


def test_reference_rounding_is_the_type_s_own():
    """The definition used by the GPU tests, against the library's cast over every border."""
    v = torch.arange(0, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double()
    half = (v[1:] + v[:-1]) / 2
    pts = torch.cat([v, half, half * (1 + 1e-6), half * (1 - 1e-6)])
    pts = torch.cat([pts, -pts])
    assert torch.equal(ref.e4m3(pts), pts.float().to(torch.float8_e4m3fn).float().double())
