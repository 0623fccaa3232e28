"""vq_fp8_quant bit for bit and vq_fp8_gemm within derived bounds against the
64-bit oracles, from one token to several tiles, odd sizes, all output types."""
import numpy as np
import pytest

from oracle import block_oracle as O
from tests.helpers import announce
from vq_dequant_matmul_gemv_amd import synth

pytestmark = pytest.mark.gpu


def _torch_dt(name):
    import torch
    return getattr(torch, name)


# ---- quantizer ------------------------------------------------------------

def _quant_check(x):
    """x: fp16 / bf16 torch tensor on the CPU."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    T, C = x.shape
    announce("fp8_quant", (T, C), str(x.dtype))
    kb = -(-C // 128)
    q = torch.full(((T + 1) * C,), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full(((T + 1) * kb,), 555.0, device="cuda")
    binding.fp8_quant(x.cuda(), q=q[:T * C].view(T, C).view(torch.float8_e4m3fn), scales=s[:T * kb].view(T, kb))
    torch.cuda.synchronize()
    rq, rs = O.fp8_quant(x.double().numpy())
    gq, gs = q[:T * C].view(T, C).cpu().numpy(), s[:T * kb].view(T, kb).cpu().numpy()
    assert np.array_equal(gs.view(np.uint32), rs.view(np.uint32))
    nan = (rq & 0x7f) == 0x7f
    assert np.array_equal((gq & 0x7f) == 0x7f, nan)
    assert np.array_equal(gq[~nan], rq[~nan]), np.argwhere((gq != rq) & ~nan)[:5]
    assert torch.all(q[T * C:] == 0x55).item() and torch.all(s[T * kb:] == 555.0).item()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("T,C", [(1, 16), (3, 112), (1, 128), (5, 144), (2, 5120), (17, 2000), (700, 384), (4, 17408)])
def test_quant_random(dtype, T, C):
    import torch
    g = synth.rng("fp8-quant", T, C)
    x = g.normal(size=(T, C)) * np.exp(g.normal(size=(T, 1)) * 3)
    x[:, :: 37] *= 20
    _quant_check(torch.from_numpy(x).to(_torch_dt(dtype)))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_quant_ties_and_grid(dtype):
    """amax a power of two times 1.75 (an exact scale): values on the e4m3 grid
    and on its ties; and amax values whose quotients lie next to ties."""
    import torch
    grid = O.E4M3[:127]
    ties = (grid[1:] + grid[:-1]) / 2
    v = np.concatenate([grid, ties, -grid, -ties, np.linspace(0, 2 ** -8, 60)])
    v = np.pad(v, (0, -len(v) % 127)).reshape(-1, 127)
    v = np.concatenate([np.full((v.shape[0], 1), 448.0), v], axis=1)
    rows = [v * 2.0 ** k for k in (0, -4, 6)]
    g = synth.rng("fp8-ties", 1)
    near = g.integers(1, 256, size=(200, 128)).astype(np.float64)     # 8-bit integers: many near ties
    _quant_check(torch.from_numpy(np.concatenate(rows + [near])).to(_torch_dt(dtype)))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_quant_extremes(dtype):
    """Zero blocks, signed zeros, the type's smallest and largest values, NaN
    and infinities beside ordinary values and alone."""
    import torch
    dt = _torch_dt(dtype)
    fi = torch.finfo(dt)
    g = synth.rng("fp8-extreme", 2)
    x = torch.from_numpy(g.normal(size=(12, 256))).to(dt)
    x[0] = 0.0
    x[1, :128] = -0.0
    x[2] = torch.from_numpy(g.integers(-9, 10, 256)).to(dt) * fi.smallest_normal / 8
    x[3] = 0
    x[3, 7] = fi.smallest_normal * fi.eps                      # one smallest subnormal
    x[4] = x[4] * fi.smallest_normal
    x[5, 3], x[5, 200] = fi.max, -fi.max
    x[6, 9] = float("nan")
    x[7, 0], x[7, 130] = float("inf"), -float("inf")
    x[8] = float("nan")
    x[9, :128] = float("inf")
    x[10, 5], x[10, 6], x[10, 7] = float("nan"), float("inf"), fi.max
    _quant_check(x)


# ---- product --------------------------------------------------------------

def _operands(T, R, C, key, spread=1.0):
    g = synth.rng("fp8-op", *key)
    kb, rb = -(-C // 128), -(-R // 128)
    xc = O.e4m3_nearest(g.normal(size=(T, C)) * 60)
    wc = O.e4m3_nearest(g.normal(size=(R, C)) * 60)
    xs = (np.exp(g.normal(size=(T, kb)) * spread) / 60).astype(np.float32)
    ws = (0.02 * np.exp(g.normal(size=(rb, kb)) * spread) / 60).astype(np.float32)
    return xc, xs, wc, ws


def _eps(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


def _product_check(ops, dtype="float32", epilogue=None, finite_only=True, stream=None):
    """Bounds: the 128 products of a block are exact and their sum rounds (or
    cuts) at most 128 times to 2^-23 of the magnitudes' sum; the scale product
    and its use round twice, and the blocks' sums kb times to 2^-24.  For 16-bit
    outputs the e4m3 instructions cut every product of a group of eight below
    2^-13 of the group's largest one, which itself (8 bits) stays whole: at most
    7 * 2^-13 of a group's magnitudes.  The output type adds half a unit, SwiGLU the usual product rule with |silu'|
    <= 1.1 and 16 units for its exp and quotient."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    xc, xs, wc, ws = ops
    (T, C), R = xc.shape, wc.shape[0]
    announce("fp8_gemm", T, R, C, dtype, epilogue)
    dt = _torch_dt(dtype)
    w = binding.FP8Tensor(torch.from_numpy(wc).cuda(), torch.from_numpy(ws).cuda())
    x, s = torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda()
    yc = R // 2 if epilogue else R
    buf = torch.full(((T + 1) * yc + 64,), 99.0, dtype=dt, device="cuda")
    y = binding.fp8_gemm(w, x.view(torch.float8_e4m3fn), s, y=buf[:T * yc].view(T, yc), epilogue=epilogue)
    torch.cuda.synchronize()
    ref, mag = O.fp8_product(xc, xs, wc, ws)
    err = mag * (128 * 2.0 ** -23 + (xs.shape[1] + 4) * 2.0 ** -24)
    if dtype != "float32":
        err = err + mag * 7 * 2.0 ** -13
    if epilogue:
        a, b, ea, eb = ref[:, 0::2], ref[:, 1::2], err[:, 0::2], err[:, 1::2]
        silu = a / (1 + np.exp(-a))
        ref = silu * b
        err = 1.1 * ea * (np.abs(b) + eb) + np.abs(silu) * eb + 16 * 2.0 ** -24 * np.abs(ref)
    got = y.double().cpu().numpy()
    tiny = float(torch.finfo(dt).smallest_normal) * _eps(dt) * 2
    tol = err + _eps(dt) * (np.abs(ref) + err) + tiny
    bad = ~(np.abs(got - ref) <= tol)
    if not finite_only:
        bad &= ~(np.isnan(ref) & np.isnan(got))
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - ref)[bad][:4], tol[bad][:4])
    assert torch.all(buf[T * yc:] == 99.0).item()
    return y


@pytest.mark.parametrize("T", [1, 2, 3, 15, 16, 17, 33, 64, 65, 100, 127, 128, 129, 200, 257, 300])
@pytest.mark.parametrize("R,C", [(64, 128), (1, 16), (129, 144), (257, 2000), (512, 1024)])
def test_product_sizes(T, R, C):
    _product_check(_operands(T, R, C, ("sizes", T, R, C)))


@pytest.mark.parametrize("T,R,C", [(1, 17408, 512), (4, 1000, 17408), (16, 5120, 5120), (513, 1030, 1008),
                                   (1024, 768, 640), (40, 4096, 4096), (300, 5120, 256), (1, 7, 17408)])
def test_product_larger(T, R, C):
    _product_check(_operands(T, R, C, ("larger", T, R, C)))


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("epilogue", [None, "swiglu"])
@pytest.mark.parametrize("T,R,C", [(1, 258, 384), (7, 514, 528), (50, 130, 256), (140, 1022, 512), (280, 384, 272)])
def test_product_types_and_swiglu(dtype, epilogue, T, R, C):
    _product_check(_operands(T, R, C, ("types", T, R, C)), dtype, epilogue)


@pytest.mark.parametrize("T", [1, 20, 150])
def test_nan_codes_stay_in_their_token_and_row(T):
    """A NaN code in x spoils that token, one in w that row, and nothing else."""
    xc, xs, wc, ws = _operands(T, 200, 400, ("nan", T))
    xc[T // 2, 77] = 0x7f
    wc[131, 399] = 0xff
    y = _product_check((xc, xs, wc, ws), finite_only=False).cpu().numpy()
    nan = np.isnan(y)
    want = np.zeros_like(nan)
    want[T // 2] = True
    want[:, 131] = True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("T", [1, 18, 140])
def test_exact_sums_are_exact(T):
    """Small integers with scales of one: every sum is exact in any order."""
    g = synth.rng("fp8-int", T)
    R, C = 300, 4096
    xi, wi = g.integers(-3, 4, (T, C)), g.integers(-3, 4, (R, C))
    xc, wc = O.e4m3_nearest(xi), O.e4m3_nearest(wi)
    ones = np.ones((T, C // 128), np.float32), np.ones((3, C // 128), np.float32)
    y = _product_check((xc, ones[0], wc, ones[1]))
    assert np.array_equal(y.cpu().numpy(), (xi @ wi.T).astype(np.float32))


@pytest.mark.parametrize("T,R,C", [(1, 512, 2048), (90, 640, 4096), (260, 700, 2048)])
def test_same_bits_again_other_stream_and_captured(T, R, C):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    xc, xs, wc, ws = _operands(T, R, C, ("again", T))
    w = binding.FP8Tensor(torch.from_numpy(wc).cuda().view(torch.float8_e4m3fn), torch.from_numpy(ws).cuda())
    x, s = torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda()
    ref = binding.fp8_gemm(w, x, s)
    assert torch.equal(ref, binding.fp8_gemm(w, x, s))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = binding.fp8_gemm(w, x, s, stream=st)
    st.synchronize()
    assert torch.equal(ref, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = binding.fp8_gemm(w, x, s)
    for k in range(3):
        x.copy_(torch.from_numpy(_operands(T, R, C, ("replay", k))[0]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, binding.fp8_gemm(w, x, s))


def test_quantize_then_multiply_a_swiglu_mlp():
    """An 8-bit MLP as it is used: quantize, gate/up with SwiGLU, quantize,
    down; each step against the oracle on the values that reached it."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    H, I, T = 512, 768, 37
    g = synth.rng("fp8-mlp")
    x = torch.from_numpy(g.normal(size=(T, H))).to(torch.bfloat16).cuda()
    _, _, gc, gs = _operands(1, 2 * I, H, ("mlp-gate-up",))
    _, _, dc, ds = _operands(1, H, I, ("mlp-down",))
    q, s = binding.fp8_quant(x)
    act = _product_check((q.view(torch.uint8).cpu().numpy(), s.cpu().numpy(), gc, gs), "bfloat16", "swiglu")
    q2, s2 = binding.fp8_quant(act)
    rq, rs = O.fp8_quant(act.double().cpu().numpy())
    assert np.array_equal(q2.view(torch.uint8).cpu().numpy(), rq) and np.array_equal(s2.cpu().numpy(), rs)
    _product_check((q2.view(torch.uint8).cpu().numpy(), s2.cpu().numpy(), dc, ds), "float32")


def test_empty_batch():
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    w = binding.FP8Tensor(torch.zeros(32, 64, dtype=torch.uint8, device="cuda"), torch.ones(1, 1, device="cuda"))
    x = torch.zeros(0, 64, dtype=torch.float16, device="cuda")
    q, s = binding.fp8_quant(x)
    assert q.shape == (0, 64) and s.shape == (0, 1)
    assert binding.fp8_gemm(w, q, s).shape == (0, 32)


# ---- every kernel and split, whatever the planner would choose -------------

KERNELS = 12


@pytest.mark.parametrize("kernel", range(KERNELS))
@pytest.mark.parametrize("splits", [1, 2, 5])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_every_kernel_and_split(kernel, splits, dtype, monkeypatch):
    """Sizes around each kernel's tile, odd rows and columns, fewer steps than
    waves, splits that leave a short last part, SwiGLU behind a split."""
    monkeypatch.setenv("VQMI_FP8_PLAN", f"{kernel},{splits}")
    for T, R, C, epi in [(1, 16, 16, None), (1, 130, 1296, "swiglu"), (17, 257, 2000, None), (65, 126, 3200, "swiglu"),
                         (191, 259, 1152, None), (193, 300, 528, None), (257, 514, 640, "swiglu")]:
        if kernel < 3 and T > 193:
            continue
        _product_check(_operands(T, R, C, ("kernel", T, R, C)), dtype, epi)


@pytest.mark.parametrize("kernel", range(KERNELS))
def test_every_kernel_on_long_rows(kernel, monkeypatch):
    """More column blocks than a chunk of scales holds, unsplit and split."""
    for splits in (1, 3):
        monkeypatch.setenv("VQMI_FP8_PLAN", f"{kernel},{splits}")
        for dtype in ("float32", "float16"):
            _product_check(_operands(18, 40, 128 * 300 + 16, ("long",), 0.2), dtype)


def test_the_planner_splits_and_its_workspace_is_enough(monkeypatch):
    """A shape the planner splits: two calls in a row on one poisoned workspace
    of exactly the stated size, with a guard behind it."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    T, R, C = 40, 640, 17408
    need = binding.LIB.vq_fp8_workspace_bytes(R, C, T)
    assert need > 0
    xc, xs, wc, ws = _operands(T, R, C, ("ws",))
    w = binding.FP8Tensor(torch.from_numpy(wc).cuda(), torch.from_numpy(ws).cuda())
    x, s = torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda()
    buf = torch.full((need + 256,), 0xff, dtype=torch.uint8, device="cuda")
    ref, _ = O.fp8_product(xc, xs, wc, ws)
    for dt in (torch.float32, torch.bfloat16):
        y = binding.fp8_gemm(w, x, s, workspace=buf[:need], y_dtype=dt)
        again = binding.fp8_gemm(w, x, s, workspace=buf[:need], y_dtype=dt)
        torch.cuda.synchronize()
        assert torch.equal(y, again) and torch.all(buf[need:] == 0xff).item()
        assert np.abs(y.double().cpu().numpy() - ref).max() <= 0.01 * np.abs(ref).max()
    with pytest.raises(binding.VQError, match="workspace"):
        binding.fp8_gemm(w, x, s, workspace=buf[:16])
