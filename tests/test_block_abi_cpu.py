"""Host checks of the operators around the VQ products, without a GPU: every
refused call returns before anything is enqueued."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def b():
    from vq_dequant_matmul_gemv_amd import binding
    return binding


def _status(b, st):
    return b.STATUS_NAMES[st]


# ---- routing --------------------------------------------------------------

def _route(b, T=4, logits=0x10000, ids=0x20000, weights=0x30000, **kw):
    base = dict(num_experts=64, top_k=8, score=0, logits_dtype=0, groups=1, top_groups=1, group_score=0,
                renormalize=1, scale=1.0, reserved=0, bias=None)
    base.update(kw)
    r = b.CRouter(**base)
    return _status(b, b.LIB.vq_moe_route(ctypes.byref(r), logits, T, ids, weights, None))


@pytest.mark.parametrize("kw,status", [
    (dict(num_experts=0), "VQ_ERR_SHAPE"),
    (dict(num_experts=1025), "VQ_ERR_SHAPE"),
    (dict(top_k=0), "VQ_ERR_SHAPE"),
    (dict(top_k=65, num_experts=128), "VQ_ERR_SHAPE"),
    (dict(top_k=9, num_experts=8), "VQ_ERR_SHAPE"),
    (dict(groups=0), "VQ_ERR_SHAPE"),
    (dict(groups=3), "VQ_ERR_SHAPE"),                        # does not divide 64
    (dict(groups=128, num_experts=1024), "VQ_ERR_SHAPE"),
    (dict(groups=8, top_groups=9), "VQ_ERR_SHAPE"),
    (dict(groups=8, top_groups=0), "VQ_ERR_SHAPE"),
    (dict(groups=16, top_groups=1), "VQ_ERR_SHAPE"),         # 4 experts left for top_k = 8
    (dict(top_groups=2), "VQ_ERR_SHAPE"),                    # groups = 1
    (dict(score=2), "VQ_ERR_SHAPE"),
    (dict(group_score=-1), "VQ_ERR_SHAPE"),
    (dict(logits_dtype=3), "VQ_ERR_SHAPE"),
    (dict(renormalize=2), "VQ_ERR_SHAPE"),
    (dict(scale=float("nan")), "VQ_ERR_SHAPE"),
    (dict(scale=float("inf")), "VQ_ERR_SHAPE"),
    (dict(reserved=1), "VQ_ERR_SHAPE"),
    (dict(T=-1), "VQ_ERR_SHAPE"),
    (dict(T=(1 << 30) + 1), "VQ_ERR_SHAPE"),
    (dict(T=1 << 30, num_experts=1024 + 0, top_k=1), None),  # 2^40 logits: the largest size taken (T = 0 below)
    (dict(logits=0), "VQ_ERR_NULL"),
    (dict(ids=0), "VQ_ERR_NULL"),
    (dict(weights=0), "VQ_ERR_NULL"),
    (dict(logits=0x10002), "VQ_ERR_ALIGN"),
    (dict(logits=0x10001, logits_dtype=2), "VQ_ERR_ALIGN"),
    (dict(ids=0x20002), "VQ_ERR_ALIGN"),
    (dict(weights=0x30001), "VQ_ERR_ALIGN"),
    (dict(bias=0x40002), "VQ_ERR_ALIGN"),
])
def test_route_refuses(b, kw, status):
    if status is None:
        kw = dict(kw, T=0)
        status = "VQ_OK"
    assert _route(b, **kw) == status, b.LIB.vq_last_error()


def test_route_null_descriptor_and_empty(b):
    assert _status(b, b.LIB.vq_moe_route(None, 0x10000, 1, 0x20000, 0x30000, None)) == "VQ_ERR_NULL"
    assert _route(b, T=0, logits=0, ids=0, weights=0) == "VQ_OK"


def test_route_wrapper_refuses_before_the_library(b):
    import torch
    r = b.Router(8, 2)
    with pytest.raises(ValueError, match="GPU"):
        b.moe_route(r, torch.zeros(3, 8))
    with pytest.raises(ValueError, match="logits must be"):
        b.moe_route(r, torch.zeros(3, 9))
    with pytest.raises(ValueError, match="score"):
        b.moe_route(b.Router(8, 2, score="relu"), torch.zeros(3, 8))
    with pytest.raises(ValueError, match="group_score"):
        b.moe_route(b.Router(8, 2, group_score="mean"), torch.zeros(3, 8))


# ---- the routing oracle's own pins ----------------------------------------

def test_route_oracle_by_hand():
    import numpy as np
    from oracle.block_oracle import route
    ln = np.log
    x = np.array([[ln(1.0), ln(4.0), ln(3.0), ln(2.0)],
                  [5.0, 5.0, 5.0, 5.0],
                  [-np.inf, np.nan, 0.0, -np.inf],
                  [-np.inf] * 4])
    ids, w = route(x, 2, renormalize=False)
    assert ids.tolist() == [[1, 2], [0, 1], [2, -1], [-1, -1]]
    assert np.allclose(w, [[0.4, 0.3], [0.25, 0.25], [1.0, 0.0], [0.0, 0.0]])
    ids, w = route(x[:1], 2, scale=3.0)
    assert np.allclose(w, [[3 * 4 / 7, 3 * 3 / 7]])
    # a bias moves the choice, not the weights; two groups, one stays
    ids, w = route(x[:1], 1, bias=[1.0, 0, 0, 0], renormalize=False)
    assert ids.tolist() == [[0]] and np.allclose(w, [[0.1]])
    ids, _ = route(x[:1], 2, groups=2, top_groups=1, group_score="max")
    assert ids.tolist() == [[1, 0]]
    ids, _ = route(x[:1], 2, groups=2, top_groups=1, group_score="top2")       # tie 5 : 5, the lowest group
    assert ids.tolist() == [[1, 0]]
    ids, w = route(np.array([[0.0, -np.inf]]), 1, score="sigmoid", renormalize=False)
    assert ids.tolist() == [[0]] and w.tolist() == [[0.5]]
