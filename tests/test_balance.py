"""Refusals of the balance loss, on the host before anything is enqueued."""
import ctypes

import pytest

from sparse_mixture_experts_amd import moe

A = 1 << 20  # a fake, 16-byte aligned device address; never dereferenced here


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def desc(**kw):
    return moe.make_desc(**{**dict(d_model=128, d_ff=64, n_experts=16, top_k=4), **kw})


FORWARD = dict(T=8, x=A, w_router=A, router_bias=A, topk_idx=A, token_mask=A, n_seqs=2, seq_off=A, logits=A,
               expert_counts=A, seq_tokens=A, prob_mean=A, loss=A, ws=A, ws_bytes=1 << 30)
BACKWARD = dict(T=8, x=A, w_router=A, topk_idx=A, token_mask=A, n_seqs=2, seq_off=A, logits=A, expert_counts=A,
                seq_tokens=A, dloss=A, dtopk_w=A, dx=A, dw_router=A, drouter_bias=A, ws=A, ws_bytes=1 << 30)
SHARED = [dict(T=-1), dict(T=(1 << 20) + 1), dict(x=None), dict(x=A + 8), dict(w_router=None), dict(topk_idx=None),
          dict(topk_idx=A + 4), dict(token_mask=A + 1), dict(n_seqs=0), dict(n_seqs=4097), dict(seq_off=None),
          dict(seq_off=A + 4), dict(logits=None), dict(expert_counts=None), dict(seq_tokens=None), dict(ws=None),
          dict(ws=A + 8)]


@pytest.mark.parametrize("change", SHARED + [dict(prob_mean=None), dict(loss=None), dict(loss=A + 4),
                                             dict(router_bias=A + 4)])
def test_forward_refusals(lib, change):
    d = desc()
    assert lib.moe_balance_loss(ctypes.byref(d), *{**FORWARD, **change}.values(), None) == moe.MOE_E_INVALID


@pytest.mark.parametrize("change", SHARED + [dict(dx=None, dw_router=None, drouter_bias=None), dict(dx=A + 4),
                                             dict(dw_router=A + 8), dict(drouter_bias=A + 2), dict(dloss=A + 4),
                                             dict(dtopk_w=A + 8)])
def test_backward_refusals(lib, change):
    d = desc()
    assert lib.moe_balance_loss_backward(ctypes.byref(d), *{**BACKWARD, **change}.values(), None) == \
        moe.MOE_E_INVALID


def test_descriptor_and_workspace(lib):
    d = desc()
    need = moe.moe_balance_workspace_size(d, 8, 2)
    assert lib.moe_balance_loss(ctypes.byref(d), *{**FORWARD, "ws_bytes": need - 1}.values(), None) == \
        moe.MOE_E_WORKSPACE
    assert lib.moe_balance_loss_backward(ctypes.byref(d), *{**BACKWARD, "ws_bytes": need - 1}.values(), None) == \
        moe.MOE_E_WORKSPACE
    bad = desc()
    bad.top_k = 17
    assert lib.moe_balance_loss(ctypes.byref(bad), *FORWARD.values(), None) == moe.MOE_E_INVALID
    assert lib.moe_balance_loss(None, *FORWARD.values(), None) == moe.MOE_E_INVALID
    size = ctypes.c_size_t()
    for T, n in ((-1, 1), (8, 0), (8, 4097)):
        assert lib.moe_balance_workspace_size(ctypes.byref(d), T, n, ctypes.byref(size)) == moe.MOE_E_INVALID
    assert lib.moe_balance_workspace_size(ctypes.byref(d), 8, 1, None) == moe.MOE_E_INVALID
    assert moe.moe_balance_workspace_size(d, 0, 1) > 0
