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


# ---- e4m3 tensors ---------------------------------------------------------

def _quant(b, x=0x10000, dtype=2, T=4, cols=256, q=0x20000, scales=0x30000):
    return _status(b, b.LIB.vq_fp8_quant(x, dtype, T, cols, q, scales, None))


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), "VQ_ERR_SHAPE"), (dict(dtype=3), "VQ_ERR_SHAPE"),
    (dict(cols=0), "VQ_ERR_SHAPE"), (dict(cols=8), "VQ_ERR_SHAPE"), (dict(cols=136 + 1), "VQ_ERR_SHAPE"),
    (dict(cols=(1 << 20) + 16), "VQ_ERR_SHAPE"), (dict(T=-1), "VQ_ERR_SHAPE"),
    (dict(T=1 << 30, cols=256), "VQ_ERR_SHAPE"),             # 2^31 blocks
    (dict(x=0), "VQ_ERR_NULL"), (dict(q=0), "VQ_ERR_NULL"), (dict(scales=0), "VQ_ERR_NULL"),
    (dict(x=0x10008), "VQ_ERR_ALIGN"), (dict(q=0x20008), "VQ_ERR_ALIGN"), (dict(scales=0x30002), "VQ_ERR_ALIGN"),
    (dict(T=0, x=0, q=0, scales=0), "VQ_OK"),
])
def test_quant_refuses(b, kw, status):
    assert _quant(b, **kw) == status, b.LIB.vq_last_error()


def _fp8(b, T=4, x=0x40000, xs=0x50000, y=0x60000, ws=0x70000, ws_bytes=1 << 40, io=None, **kw):
    base = dict(values=0x10000, scales=0x20000, rows=300, cols=272)
    base.update(kw)
    base.setdefault("value_bytes", base["rows"] * base["cols"])
    base.setdefault("scale_elems", -(-base["rows"] // 128) * -(-base["cols"] // 128))
    w = b.CFP8Tensor(**base)
    i = None if io is None else ctypes.byref(b.CIo(*io))
    return _status(b, b.LIB.vq_fp8_gemm(ctypes.byref(w), i, x, xs, T, y, ws, ws_bytes, None))


@pytest.mark.parametrize("kw,status", [
    (dict(values=0), "VQ_ERR_NULL"), (dict(scales=0), "VQ_ERR_NULL"),
    (dict(x=0), "VQ_ERR_NULL"), (dict(xs=0), "VQ_ERR_NULL"), (dict(y=0), "VQ_ERR_NULL"),
    (dict(rows=0), "VQ_ERR_SHAPE"), (dict(rows=(1 << 24) + 1), "VQ_ERR_SHAPE"),
    (dict(cols=8), "VQ_ERR_SHAPE"), (dict(cols=280), "VQ_ERR_SHAPE"), (dict(cols=-16), "VQ_ERR_SHAPE"),
    (dict(T=-1), "VQ_ERR_SHAPE"), (dict(T=(1 << 24) + 1), "VQ_ERR_SHAPE"),
    (dict(T=1 << 24, rows=1 << 24), "VQ_ERR_SHAPE"),
    (dict(value_bytes=300 * 272 - 16), "VQ_ERR_SHAPE"),
    (dict(scale_elems=8), "VQ_ERR_SHAPE"),                    # a slice of the scales
    (dict(values=0x10008), "VQ_ERR_ALIGN"), (dict(scales=0x20002), "VQ_ERR_ALIGN"),
    (dict(x=0x40008), "VQ_ERR_ALIGN"), (dict(xs=0x50001), "VQ_ERR_ALIGN"), (dict(y=0x60008), "VQ_ERR_ALIGN"),
    (dict(io=(1, 0, 0, 0, None)), "VQ_ERR_SHAPE"),            # x_dtype is not e4m3
    (dict(io=(3, 3, 0, 0, None)), "VQ_ERR_SHAPE"),            # y cannot be e4m3
    (dict(io=(3, 0, 2, 0, None)), "VQ_ERR_SHAPE"),            # COMBINE
    (dict(io=(3, 0, 0, 1, None)), "VQ_ERR_SHAPE"),            # reserved
    (dict(io=(3, 0, 1, 0, None), rows=301), "VQ_ERR_SHAPE"),  # SWIGLU on odd rows
    (dict(T=0, x=0, xs=0, y=0, ws=0, ws_bytes=0), "VQ_OK"),
])
def test_fp8_gemm_refuses(b, kw, status):
    assert _fp8(b, **kw) == status, b.LIB.vq_last_error()


def test_fp8_workspace(b):
    """The size is a pure function of the sizes; a call that needs some and
    gets less, none or a misaligned one is refused."""
    assert b.LIB.vq_fp8_workspace_bytes(300, 272, 0) == 0
    assert b.LIB.vq_fp8_workspace_bytes(300, 8, 4) == 0 and b"cols" in b.LIB.vq_last_error()
    for T, rows, cols in [(1, 17408, 5120), (64, 512, 17408), (100, 5120, 17408), (200, 256, 4096), (2048, 5120, 17408)]:
        need = b.LIB.vq_fp8_workspace_bytes(rows, cols, T)
        if need:
            kw = dict(T=T, rows=rows, cols=cols)
            assert _fp8(b, ws=0, ws_bytes=need, **kw) == "VQ_ERR_WORKSPACE"
            assert _fp8(b, ws_bytes=need - 1, **kw) == "VQ_ERR_WORKSPACE"
            assert _fp8(b, ws=0x70008, ws_bytes=need, **kw) == "VQ_ERR_ALIGN"


def test_fp8_wrapper_refuses_before_the_library(b):
    import torch
    x = torch.zeros(3, 32, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        b.fp8_quant(x)
    with pytest.raises(ValueError, match="fp16 or bf16"):
        b.fp8_quant(x.float())
    with pytest.raises(ValueError, match="GPU"):
        b.FP8Tensor(torch.zeros(8, 32, dtype=torch.uint8), torch.ones(1, 1)).cstruct()


def test_e4m3_oracle_matches_the_type(b):
    """The oracle's code table and rounding against torch's conversion."""
    import numpy as np
    import torch
    from oracle import block_oracle as O
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(table, O.E4M3, equal_nan=True)
    v = np.random.default_rng(3).normal(size=4000).astype(np.float32) * 60
    v = np.concatenate([v, O.E4M3[:127], (O.E4M3[1:127] + O.E4M3[:126]) / 2, v * 2.0 ** -12]).astype(np.float32)
    want = torch.from_numpy(np.clip(v, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.e4m3_nearest(v), want)


# ---- norms ----------------------------------------------------------------

def _norm(b, T=4, block=0x10000, residual=0x20000, v=0x30000, h=0x40000, hs=0x50000, **kw):
    base = dict(cols=256, block_dtype=0, residual_dtype=2, weight_dtype=2, h_dtype=2, gate=0, gate_act=0, reserved=0,
                alpha=1.0, beta=1.0, eps=1e-6, weight_offset=0.0, post_weight=0x60000, pre_weight=0x70000,
                gate_values=0x80000)
    base.update(kw)
    n = b.CNormSpec(**base)
    return _status(b, b.LIB.vq_norm(ctypes.byref(n), block, residual, T, v, h, hs, None))


@pytest.mark.parametrize("kw,status", [
    (dict(cols=0), "VQ_ERR_SHAPE"), (dict(cols=32769), "VQ_ERR_SHAPE"),
    (dict(block_dtype=3), "VQ_ERR_SHAPE"), (dict(residual_dtype=3), "VQ_ERR_SHAPE"),
    (dict(weight_dtype=-1), "VQ_ERR_SHAPE"), (dict(h_dtype=4), "VQ_ERR_SHAPE"),
    (dict(h_dtype=3, cols=248), "VQ_ERR_SHAPE"),
    (dict(gate=4), "VQ_ERR_SHAPE"), (dict(gate=1, gate_act=3), "VQ_ERR_SHAPE"), (dict(gate_act=1), "VQ_ERR_SHAPE"),
    (dict(eps=-1.0), "VQ_ERR_SHAPE"), (dict(eps=float("nan")), "VQ_ERR_SHAPE"),
    (dict(alpha=float("inf")), "VQ_ERR_SHAPE"), (dict(beta=float("nan")), "VQ_ERR_SHAPE"),
    (dict(weight_offset=float("inf")), "VQ_ERR_SHAPE"), (dict(reserved=1), "VQ_ERR_SHAPE"),
    (dict(T=-1), "VQ_ERR_SHAPE"), (dict(T=(1 << 30) + 1), "VQ_ERR_SHAPE"),
    (dict(block=0), "VQ_ERR_SHAPE"),                            # a post norm without a block
    (dict(block=0, post_weight=0, gate=1), "VQ_ERR_SHAPE"),
    (dict(block=0, residual=0, post_weight=0), "VQ_ERR_NULL"),
    (dict(v=0, h=0), "VQ_ERR_NULL"),
    (dict(gate=2, gate_values=0), "VQ_ERR_NULL"),
    (dict(h_dtype=3, hs=0), "VQ_ERR_NULL"),
    (dict(block=0x10008), "VQ_ERR_ALIGN"), (dict(residual=0x20008), "VQ_ERR_ALIGN"),
    (dict(v=0x30004), "VQ_ERR_ALIGN"), (dict(h=0x40002), "VQ_ERR_ALIGN"),
    (dict(post_weight=0x60008), "VQ_ERR_ALIGN"), (dict(pre_weight=0x70002), "VQ_ERR_ALIGN"),
    (dict(gate=1, gate_values=0x80008), "VQ_ERR_ALIGN"), (dict(gate=2, gate_values=0x80001), "VQ_ERR_ALIGN"),
    (dict(hs=0x50002), "VQ_ERR_ALIGN"),
    (dict(T=0, block=0, residual=0, v=0, h=0), "VQ_OK"),
])
def test_norm_refuses(b, kw, status):
    assert _norm(b, **kw) == status, b.LIB.vq_last_error()


def test_norm_wrapper_refuses_before_the_library(b):
    import torch
    x = torch.zeros(3, 32)
    with pytest.raises(ValueError, match="needs a block or a residual"):
        b.norm()
    with pytest.raises(ValueError, match="GPU"):
        b.norm(x)
    with pytest.raises(ValueError, match="nothing to compute"):
        b.norm(x, store_residual=False)


def test_packed_descriptors_have_the_structures_layout(b):
    """The bytes the wrappers pass are the ctypes mirrors' (and the header's)."""
    r = b.CRouter(256, 8, 1, 2, 8, 4, 1, 1, 2.5, 0, 0x1234567890)
    assert bytes(r) == b._pack_router(256, 8, 1, 2, 8, 4, 1, True, 2.5, 0, 0x1234567890)
    w = b.CFP8Tensor(0x1000, 0x2000, 7, 16, 112, 1)
    assert bytes(w) == b._pack_fp8(0x1000, 0x2000, 7, 16, 112, 1)
    io = b.CIo(3, 2, 1, 0, None)
    assert bytes(io) == b._pack_io(3, 2, 1, 0, 0)
    n = b.CNormSpec(64, 0, 1, 2, 3, 1, 2, 0, 0.5, 0.25, 1e-6, 1.0, 0x10, 0x20, 0x30)
    assert bytes(n) == b._pack_norm(64, 0, 1, 2, 3, 1, 2, 0, 0.5, 0.25, 1e-6, 1.0, 0x10, 0x20, 0x30)


# ---- launches of 2^32 threads and more are refused -------------------------

def test_calls_too_large_for_a_launch_are_refused(b):
    assert _route(b, T=(1 << 25) + 1) == "VQ_ERR_SHAPE"
    assert _status(b, b.LIB.vq_fp8_quant(0x10000, 1, 1 << 28, 128, 0x20000, 0x30000, None)) == "VQ_ERR_SHAPE"
    assert _status(b, b.LIB.vq_fp8_quant(0x10000, 1, 1 << 27, 256, 0x20000, 0x30000, None)) == "VQ_ERR_SHAPE"
    for T, cols in [(1 << 26, 8), (1 << 25, 513), (1 << 20, 32768)]:
        spec = b.CNormSpec(cols=cols, block_dtype=0, residual_dtype=0, weight_dtype=0, h_dtype=0, gate=0, gate_act=0,
                           reserved=0, alpha=1.0, beta=1.0, eps=1e-6, weight_offset=0.0)
        assert _status(b, b.LIB.vq_norm(ctypes.byref(spec), 0x10000, 0, T, 0, 0x20000, None, None)) == "VQ_ERR_SHAPE"


# ---- the product with the e4m3 instructions allowed ------------------------

def test_fast_fp8_gemm_refuses_an_fp32_y_and_what_the_exact_one_refuses(b):
    w = b.CFP8Tensor(values=0x10000, scales=0x20000, rows=300, cols=272, value_bytes=300 * 272, scale_elems=9)

    def call(io, T=4, x=0x40000):
        i = None if io is None else ctypes.byref(b.CIo(*io))
        return _status(b, b.LIB.vq_fp8_gemm_fast(ctypes.byref(w), i, x, 0x50000, T, 0x60000, 0x70000, 1 << 40, None))

    assert call(None) == "VQ_ERR_SHAPE" and b"F16 or BF16" in b.LIB.vq_last_error()
    assert call((3, 0, 0, 0, None)) == "VQ_ERR_SHAPE"
    assert call((3, 2, 2, 0, None)) == "VQ_ERR_SHAPE"                       # COMBINE
    assert call((3, 1, 0, 0, None), x=0x40008) == "VQ_ERR_ALIGN"
    assert call((3, 1, 0, 0, None), T=-1) == "VQ_ERR_SHAPE" and b"vq_fp8_gemm_fast" in b.LIB.vq_last_error()
    assert call((3, 2, 1, 0, None), T=0) == "VQ_OK"


def test_the_largest_sizes_taken_and_the_first_ones_refused(b):
    """Grids round up to whole blocks and still hold fewer than 2^32 threads.  A
    size that is taken fails on the NULL outputs behind it: nothing is launched."""
    def route(T):
        return _route(b, T=T, ids=0)

    def quant(T, cols):
        return _quant(b, T=T, cols=cols, q=0)

    def norm(T, cols):
        return _norm(b, T=T, cols=cols, v=0, h=0)

    for call, taken, refused in [(route, [(1 << 25,)], [((1 << 25) + 1,)]),
                                 (quant, [((1 << 28) - 16, 16), ((1 << 27) - 8, 256), ((1 << 28) // 3 - 6, 384)],
                                  [((1 << 28) - 15, 16), ((1 << 28) - 1, 128), ((1 << 27) - 7, 256)]),
                                 (norm, [((1 << 26) - 4, 8), ((1 << 26) - 4, 511), ((1 << 25) - 2, 513), ((1 << 20) - 1, 32768)],
                                  [((1 << 26) - 3, 8), ((1 << 26) - 1, 512), ((1 << 25) - 1, 513), (1 << 20, 32768)])]:
        for a in taken:
            assert call(*a) == "VQ_ERR_NULL", (a, b.LIB.vq_last_error())
        for a in refused:
            assert call(*a) == "VQ_ERR_SHAPE", (a, b.LIB.vq_last_error())


def test_weight_scales_of_another_layout_are_refused(b):
    """[cols/128][rows/128] holds as many values as [rows/128][cols/128]: the
    shape tells them apart, before a GPU is needed."""
    import torch
    v = torch.zeros(256, 640, dtype=torch.uint8)
    x, xs = torch.zeros(3, 640, dtype=torch.uint8), torch.ones(3, 5)
    for scales in (torch.ones(5, 2), torch.ones(10), torch.ones(2, 5, 1), torch.ones(2, 4), torch.ones(2, 5).half()):
        w = b.FP8Tensor(v, scales)
        with pytest.raises(ValueError, match="w.scales must be"):
            b.fp8_gemm(w, x, xs)
        with pytest.raises(ValueError, match="w.scales must be"):
            w.cstruct()
    with pytest.raises(ValueError, match="GPU"):                 # the right shape gets as far as the device
        b.fp8_gemm(b.FP8Tensor(v, torch.ones(2, 5)), x, xs)


# ---- the product's plan -----------------------------------------------------

@pytest.mark.parametrize("T,rows", [(1 << 14, 1 << 24), (1 << 24, 1 << 14), ((1 << 14) - 128 + 1, 1 << 23 | 1)])
def test_sizes_no_kernel_holds_in_one_launch_are_refused(b, T, rows):
    """Up to 2^30 tiles of 16 x 16 pass the first check; where the largest tiles
    still make 2^22 of them there is no plan, and nothing may run in its place."""
    for call in (b.LIB.vq_fp8_gemm, b.LIB.vq_fp8_gemm_fast):
        w = b.CFP8Tensor(values=0x10000, scales=0x20000, rows=rows, cols=16, value_bytes=rows * 16,
                         scale_elems=-(-rows // 128))
        if call is b.LIB.vq_fp8_gemm_fast and T < 1 << 14:
            continue                             # 256 x 256 tiles: half as many
        io = b.CIo(3, 2, 0, 0, None)
        # the NULL x behind the check keeps a size that is taken from being launched
        st = _status(b, call(ctypes.byref(w), ctypes.byref(io), 0, 0x50000, T, 0x60000, 0x70000, 1 << 40, None))
        assert st == "VQ_ERR_SHAPE" and b"too many tiles" in b.LIB.vq_last_error()


def test_a_forced_plan_keeps_the_planners_limits(b, monkeypatch):
    """VQMI_FP8_PLAN with more planes than the planner would ever ask for (512
    MiB) is passed over; one within them is taken, and a stated workspace is what
    the call wants."""
    free = b.LIB.vq_fp8_workspace_bytes(17408, 5120, 4096)
    assert free <= 512 << 20
    monkeypatch.setenv("VQMI_FP8_PLAN", "3,8")
    assert b.LIB.vq_fp8_workspace_bytes(17408, 5120, 4096) == free
    need = b.LIB.vq_fp8_workspace_bytes(640, 5120, 64)
    assert need >= 5 * 640 * 64 * 4          # 40 column blocks in parts of whole fours: 5 of 8
    kw = dict(T=64, rows=640, cols=5120)
    assert _fp8(b, ws_bytes=need - 1, **kw) == "VQ_ERR_WORKSPACE"
    assert _fp8(b, ws=0x70008, ws_bytes=need, **kw) == "VQ_ERR_ALIGN"


def test_some_shapes_need_a_workspace(b):
    """So that the workspace checks above are made at all."""
    for T, rows, cols in [(64, 512, 17408), (40, 640, 17408), (16, 5120, 17408)]:
        assert b.LIB.vq_fp8_workspace_bytes(rows, cols, T) > 0
