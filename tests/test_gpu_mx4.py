"""vq_mx4_quant and vq_mx4_dequant bit for bit and vq_mx4_gemm within derived
bounds against the 64-bit oracles: one token to several tiles, odd sizes, scales
from one end to the other, all input and output types."""
import numpy as np
import pytest

from oracle import block_oracle as O
from tests.helpers import announce
from vq_dequant_matmul_gemv_amd import synth

pytestmark = pytest.mark.gpu


def _dt(name):
    import torch
    return getattr(torch, name)


def _eps(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


# ---- quantizer and reader -------------------------------------------------

def _quant_check(x):
    """x: CPU tensor [T][C].  Codes, scales and the values read back, with guards
    behind every output."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    T, C = x.shape
    announce("mx4_quant", (T, C), str(x.dtype))
    q = torch.full(((T + 1) * C // 2,), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full(((T + 1) * C // 32,), 0x77, dtype=torch.uint8, device="cuda")
    nq, ns = T * C // 2, T * C // 32
    binding.mx4_quant(x.cuda(), q=q[:nq].view(T, C // 2), scales=s[:ns].view(T, C // 32))
    torch.cuda.synchronize()
    rq, rs = O.mx4_quant(x.double().numpy())
    gq, gs = q[:nq].view(T, -1).cpu().numpy(), s[:ns].view(T, -1).cpu().numpy()
    assert np.array_equal(gs, rs), np.argwhere(gs != rs)[:5]
    assert np.array_equal(gq, rq), np.argwhere(gq != rq)[:5]
    assert torch.all(q[nq:] == 0x55).item() and torch.all(s[ns:] == 0x77).item()
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        _dequant_check(rq, rs, dt)


def _dequant_check(rq, rs, dt):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    T, C = rq.shape[0], rq.shape[1] * 2
    buf = torch.full(((T + 1) * C,), 7.0, dtype=dt, device="cuda")
    binding.mx4_dequant(torch.from_numpy(rq).cuda(), torch.from_numpy(rs).cuda(), y=buf[:T * C].view(T, C))
    torch.cuda.synchronize()
    want = torch.from_numpy(O.mx4_values(rq, rs)).to(dt)        # rounded once
    got = buf[:T * C].view(T, C).cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0.0, 1e4, -1e4), want.nan_to_num(0.0, 1e4, -1e4))
    assert torch.equal(torch.signbit(got) | torch.isnan(got), torch.signbit(want) | torch.isnan(want))
    assert torch.all(buf[T * C:] == 7.0).item()


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("T,C", [(1, 32), (3, 96), (1, 128), (5, 160), (2, 5120), (17, 2016), (700, 384), (4, 17408)])
def test_quant_random(dtype, T, C):
    import torch
    g = synth.rng("mx4-quant", T, C)
    x = g.normal(size=(T, C)) * np.exp(g.normal(size=(T, 1)) * 3)
    x[:, :: 37] *= 20
    _quant_check(torch.from_numpy(x).to(_dt(dtype)))


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_quant_grid_ties_and_neighbours(dtype):
    """Values on the grid, on its ties and next to them, under every largest
    value that moves the scale: powers of two, 6 and what is above it."""
    import torch
    dt = _dt(dtype)
    grid = O.E2M1[:8]
    ties = (grid[1:] + grid[:-1]) / 2
    near = [t * (1 + k * 2.0 ** -7) for t in ties for k in (-1, 1)]
    v = np.concatenate([grid, ties, near, -grid, -ties])
    v = np.pad(v, (0, -len(v) % 31)).reshape(-1, 31)
    rows = []
    for top in (4.0, 4.03125, 6.0, 7.0, 7.96875):
        for p in (0, -9, 5):
            rows.append(np.concatenate([np.full((v.shape[0], 1), top), v], axis=1) * 2.0 ** p)
    _quant_check(torch.from_numpy(np.concatenate(rows).reshape(-1, 32)).to(dt))


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_quant_extremes(dtype):
    """Zeros of both signs, the type's smallest and largest values, NaN and
    infinities beside ordinary values and alone."""
    import torch
    dt = _dt(dtype)
    fi = torch.finfo(dt)
    g = synth.rng("mx4-extreme", 2)
    x = torch.from_numpy(g.normal(size=(14, 96))).to(dt)
    x[0] = 0.0
    x[1, :40] = -0.0
    x[2] = torch.from_numpy(g.integers(-9, 10, 96)).to(dt) * fi.smallest_normal / 8
    x[3] = 0
    x[3, 7] = fi.smallest_normal * fi.eps
    x[4] = x[4] * fi.smallest_normal
    x[5, 3], x[5, 90] = fi.max, -fi.max
    x[6, 9] = float("nan")
    x[7, 0], x[7, 50] = float("inf"), -float("inf")
    x[8] = float("nan")
    x[9, :32] = float("inf")
    x[10, 5], x[10, 6], x[10, 7] = float("nan"), float("inf"), fi.max
    x[11] = fi.smallest_normal
    x[12, ::3] = fi.smallest_normal * 4
    _quant_check(x)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_dequant_every_code_and_scale(dtype):
    """Every scale byte over every code: what fp16 cannot hold rounds once."""
    codes = np.tile(np.arange(16, dtype=np.uint8), 512).reshape(256, 32)
    _dequant_check(O.mx4_pack(codes), np.arange(256, dtype=np.uint8).reshape(256, 1), _dt(dtype))


# ---- product --------------------------------------------------------------

def _operands(T, R, C, key, x="mx4", lo=119, hi=135):
    """4-bit operands of random codes with scale bytes in [lo, hi]; 16-bit
    activations with some large channels."""
    g = synth.rng("mx4-op", *key)
    pack = lambda n: (g.integers(0, 256, (n, C // 2), dtype=np.uint8),  # noqa: E731
                      g.integers(lo, hi + 1, (n, C // 32), dtype=np.uint8))
    w = pack(R)
    if x == "mx4":
        return pack(T), w
    import torch
    v = g.normal(size=(T, C)) * np.where(g.uniform(size=C) < 1 / 64, 20, 1)
    return (torch.from_numpy(v).to(_dt(x)), None), w


def _product_check(ops, y_dtype="float32", epilogue=None, guard=99.0):
    """Bounds.  Products are exact.  4-bit x: each 16 x 16 x 128 instruction is
    off by at most 4 units of 2^-24 of the largest of its block sums and its
    accumulator, which the magnitudes' sum bounds: blocks / 4 instructions.
    16-bit x: an instruction of 32 columns by at most 6 units (2 of them with
    two instructions a block where x is taken apart).  Joins of waves and column
    splits add 32.  The output type adds half a unit, SwiGLU the product rule
    with |silu'| <= 1.1 and 16 units for its exp and quotient."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    (xq, xs), (wq, ws) = ops
    R, C = wq.shape[0], wq.shape[1] * 2
    T = xq.shape[0]
    announce("mx4_gemm", T, R, C, y_dtype, epilogue, "mx4" if xs is not None else xq.dtype)
    dt = _dt(y_dtype)
    w = binding.MX4Tensor(torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda())
    if xs is not None:
        xv = O.mx4_values(xq, xs)
        args = (torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda())
    else:
        xv = xq.double().numpy()
        args = (xq.cuda(),)
    yc = R // 2 if epilogue else R
    buf = torch.full(((T + 1) * yc + 64,), guard, dtype=dt, device="cuda")
    y = binding.mx4_gemm(w, *args, y=buf[:T * yc].view(T, yc), epilogue=epilogue)
    torch.cuda.synchronize()
    wv = O.mx4_values(wq, ws)
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    units = (1 if xs is not None else 12) * (C // 32) + 36
    err = mag * units * 2.0 ** -24
    if epilogue:
        a, b, ea, eb = ref[:, 0::2], ref[:, 1::2], err[:, 0::2], err[:, 1::2]
        ref = O.swiglu(ref)
        silu = a / (1 + np.exp(-np.clip(a, -700, None)))
        err = 1.1 * ea * (np.abs(b) + eb) + np.abs(silu) * eb + 16 * 2.0 ** -24 * np.abs(ref)
    got = y.double().cpu().numpy()
    tiny = float(torch.finfo(dt).smallest_normal) * _eps(dt) * 2
    tol = err + _eps(dt) * (np.abs(ref) + err) + tiny
    # rounding to nearest makes every value from half a step above the type's
    # largest one on an infinity (fp16: from 65520), and y may be off by err
    over = np.isinf(got) & (np.sign(got) == np.sign(ref)) & \
        (np.abs(ref) + err >= float(torch.finfo(dt).max) * (1 + _eps(dt) / 2))
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - ref) <= tol) & ~(np.isnan(ref) & np.isnan(got)) & ~over
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - ref)[bad][:4], tol[bad][:4])
    assert torch.all(buf[T * yc:] == guard).item()
    return y


@pytest.mark.parametrize("T", [1, 2, 3, 15, 16, 17, 33, 64, 65, 100, 127, 128, 129, 200, 257, 300])
@pytest.mark.parametrize("R,C", [(64, 128), (1, 32), (129, 160), (257, 2016), (512, 1024)])
def test_product_sizes(T, R, C):
    _product_check(_operands(T, R, C, ("sizes", T, R, C)))


@pytest.mark.parametrize("x", ["float16", "bfloat16"])
@pytest.mark.parametrize("T", [1, 2, 16, 17, 33, 64, 65, 130, 300])
@pytest.mark.parametrize("R,C", [(64, 128), (1, 32), (129, 160), (257, 2016), (512, 1024)])
def test_product_sizes_16_bit_x(x, T, R, C):
    _product_check(_operands(T, R, C, ("sizes16", T, R, C), x))


@pytest.mark.parametrize("x", ["mx4", "float16", "bfloat16"])
@pytest.mark.parametrize("T,R,C", [(1, 17408, 512), (4, 1000, 17408), (16, 5120, 5120), (513, 1030, 1056),
                                   (1024, 768, 640), (40, 4096, 4096), (300, 5120, 256), (1, 7, 17408)])
def test_product_larger(x, T, R, C):
    _product_check(_operands(T, R, C, ("larger", T, R, C), x))


@pytest.mark.parametrize("x", ["mx4", "float16", "bfloat16"])
@pytest.mark.parametrize("y", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("epilogue", [None, "swiglu"])
@pytest.mark.parametrize("T,R,C", [(1, 258, 384), (7, 514, 544), (50, 130, 256), (140, 1022, 512), (280, 384, 288)])
def test_product_types_and_swiglu(x, y, epilogue, T, R, C):
    _product_check(_operands(T, R, C, ("types", T, R, C), x, 115, 127), y, epilogue)


@pytest.mark.parametrize("x", ["mx4", "float16", "bfloat16"])
@pytest.mark.parametrize("T,R,C", [(1, 64, 1024), (40, 100, 544), (200, 272, 2048)])
@pytest.mark.parametrize("lo,hi", [(100, 112), (134, 146), (97, 157), (127, 127)])
def test_product_scales_over_a_wide_range(x, T, R, C, lo, hi):
    """Scales whose values fp16 can hold, cannot hold, and both in one step."""
    _product_check(_operands(T, R, C, ("wide", T, lo, hi), x, lo, hi))


@pytest.mark.parametrize("x", ["float16", "bfloat16"])
@pytest.mark.parametrize("T", [1, 40, 150])
def test_product_16_bit_x_extremes(x, T):
    """The largest and smallest scales and activations: sums stay inside fp32."""
    import torch
    g = synth.rng("mx4-extreme16", T)
    C, R = 256, 48
    wq = g.integers(0, 256, (R, C // 2), dtype=np.uint8)
    ws = np.repeat(g.choice([0, 1, 20, 127, 200, 230], size=(R, 1)).astype(np.uint8), C // 32, axis=1)
    v = torch.from_numpy(g.normal(size=(T, C))).to(_dt(x))
    fi = torch.finfo(_dt(x))
    v[:, 5] = fi.smallest_normal * fi.eps if x == "float16" else fi.smallest_normal
    v[T // 2, ::2] = 65504.0 if x == "float16" else 60000.0
    _product_check(((v, None), (wq, ws)))


@pytest.mark.parametrize("T", [1, 20, 150])
@pytest.mark.parametrize("x", ["mx4", "float16", "bfloat16"])
def test_nan_stays_in_its_token_and_row(T, x):
    """A NaN scale (or a NaN value) in x spoils that token, one in w that row,
    and nothing else."""
    (xq, xs), (wq, ws) = _operands(T, 200, 416, ("nan", T), x, 120, 130)
    if x == "mx4":
        xs[T // 2, 3] = 255
    else:
        xq[T // 2, 100] = float("nan")
    ws[131, 12] = 255
    y = _product_check(((xq, xs), (wq, ws))).cpu().numpy()
    want = np.zeros_like(y, dtype=bool)
    want[T // 2] = True
    want[:, 131] = True
    assert np.array_equal(np.isnan(y), want)


@pytest.mark.parametrize("x", ["float16", "bfloat16"])
def test_infinite_activations(x):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    (xv, _), (wq, ws) = _operands(3, 32, 128, ("inf",), x, 60, 60)     # scales fp16 cannot hold
    wq[:] = 0x22
    wq[5] = 0xaa
    xv[1, 3] = float("inf")
    y = binding.mx4_gemm(binding.MX4Tensor(torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda()), xv.cuda()).cpu()
    assert torch.isfinite(y[[0, 2]]).all() and (y[1] == torch.where(torch.arange(32) == 5, -torch.inf, torch.inf)).all()


@pytest.mark.parametrize("T", [1, 18, 140, 300])
@pytest.mark.parametrize("x", ["mx4", "float16", "bfloat16"])
def test_exact_sums_are_exact(T, x):
    """Scales of one and whole activations: every sum is exact in any order."""
    import torch
    g = synth.rng("mx4-int", T)
    R, C = 300, 4096
    (xq, xs), (wq, ws) = _operands(T, R, C, ("int", T), "mx4", 127, 127)
    if x != "mx4":
        xq, xs = torch.from_numpy(g.integers(-3, 4, (T, C)).astype(np.float64)).to(_dt(x)), None
    y = _product_check(((xq, xs), (wq, ws)))
    xv = O.mx4_values(xq, xs) if x == "mx4" else xq.double().numpy()
    assert np.array_equal(y.cpu().numpy(), (xv @ O.mx4_values(wq, ws).T).astype(np.float32))


@pytest.mark.parametrize("T", [1, 40, 200])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_scales_off_their_words(T, shift):
    """Scales that start anywhere, as slices of a larger buffer do."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    (xq, xs), (wq, ws) = _operands(T, 130, 512, ("shift", T, shift))
    def moved(s):
        buf = torch.zeros(s.size + 8, dtype=torch.uint8, device="cuda")
        v = buf[shift:shift + s.size].view(s.shape)
        v.copy_(torch.from_numpy(s))
        return v
    a = torch.from_numpy(xq).cuda()
    q = torch.from_numpy(wq).cuda()
    ref = binding.mx4_gemm(binding.MX4Tensor(q, torch.from_numpy(ws).cuda()), a, torch.from_numpy(xs).cuda())
    got = binding.mx4_gemm(binding.MX4Tensor(q, moved(ws)), a, moved(xs))
    assert torch.equal(ref, got)


@pytest.mark.parametrize("x", ["mx4", "bfloat16"])
@pytest.mark.parametrize("T,R,C", [(1, 512, 2048), (16, 640, 17408), (90, 640, 4096), (260, 700, 2048)])
def test_same_bits_again_other_stream_and_captured(x, T, R, C):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    (xq, xs), (wq, ws) = _operands(T, R, C, ("again", T), x)
    w = binding.MX4Tensor(torch.from_numpy(wq).cuda().view(torch.float4_e2m1fn_x2),
                          torch.from_numpy(ws).cuda().view(torch.float8_e8m0fnu))
    a = torch.from_numpy(xq).cuda() if xs is not None else xq.cuda()
    s = None if xs is None else torch.from_numpy(xs).cuda()
    ref = binding.mx4_gemm(w, a, s)
    assert torch.equal(ref, binding.mx4_gemm(w, a, s))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(ref)
    binding.mx4_gemm(w, a, s, y=y, stream=st)
    st.synchronize()
    assert torch.equal(ref, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = binding.mx4_gemm(w, a, s)
    other = a.flip(0).contiguous() if T > 1 else a.clone()
    keep = a.clone()
    for k in range(3):
        a.copy_(other if k % 2 else keep)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, binding.mx4_gemm(w, a, s))


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("kernel", range(24))
def test_every_kernel_and_split(kernel, splits, monkeypatch):
    """Every row of the table on tiles that end in the middle, whatever the
    planner would choose."""
    monkeypatch.setenv("VQMI_MX4_PLAN", f"{kernel},{splits}")
    for x in ("mx4", "float16", "bfloat16"):
        for T, R, C in ((1, 40, 2016), (37, 300, 1184), (270, 530, 1600)):
            _product_check(_operands(T, R, C, ("every", T, R, C), x))
        _product_check(_operands(70, 258, 1664, ("every", "swiglu"), x, 115, 127), "bfloat16", "swiglu")
    (xq, xs), (wq, ws) = _operands(20, 200, 1440, ("every", "nan"))
    xs[7, 3] = 255
    ws[131, 44] = 255
    y = _product_check(((xq, xs), (wq, ws))).cpu().numpy()
    want = np.zeros_like(y, dtype=bool)
    want[7] = True
    want[:, 131] = True
    assert np.array_equal(np.isnan(y), want)


def test_quantized_chain_captured():
    """Quantize, multiply with the fused SwiGLU, quantize again, multiply: as an
    MLP runs, eager and replayed."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    g = torch.Generator(device="cuda").manual_seed(3)
    H, I, T = 512, 768, 37
    up = binding.MX4Tensor(*binding.mx4_quant(0.05 * torch.randn(2 * I, H, device="cuda", generator=g)))
    down = binding.MX4Tensor(*binding.mx4_quant(0.05 * torch.randn(H, I, device="cuda", generator=g)))
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()

    def mlp():
        h = binding.mx4_gemm(up, *binding.mx4_quant(x), y_dtype=torch.bfloat16, epilogue="swiglu")
        return h, binding.mx4_gemm(down, *binding.mx4_quant(h))

    h, y = mlp()
    hv = O.mx4_values(*(t.view(torch.uint8).cpu().numpy() for t in binding.mx4_quant(h)))
    wv = O.mx4_values(*(t.view(torch.uint8).cpu().numpy() for t in (down.values, down.scales)))
    ref, mag = hv @ wv.T, np.abs(hv) @ np.abs(wv).T
    assert (np.abs(y.double().cpu().numpy() - ref) <= mag * (I // 32 + 36) * 2.0 ** -24 + np.abs(ref) * 2.0 ** -24).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hc, yc = mlp()
    for k in range(3):
        x.copy_(torch.randn(T, H, device="cuda", generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        h, y = mlp()
        torch.cuda.synchronize()
        assert torch.equal(h, hc) and torch.equal(y, yc)


# ---- streams, workspaces, refusals ---------------------------------------

def _random_tensor(R, C, g, lo=120, hi=126):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    return binding.MX4Tensor(torch.randint(0, 256, (R, C // 2), dtype=torch.uint8, device="cuda", generator=g),
                             torch.randint(lo, hi + 1, (R, C // 32), dtype=torch.uint8, device="cuda", generator=g))


def test_two_streams_at_once():
    """Calls that overlap in time, each with a workspace of its own."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    g = torch.Generator(device="cuda").manual_seed(5)
    w = _random_tensor(640, 17408, g)
    xs = [torch.randn(T, 17408, device="cuda", generator=g).bfloat16() for T in (16, 33)]
    ref = [(binding.mx4_gemm(w, x), binding.mx4_gemm(w, *binding.mx4_quant(x))) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(6):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append((binding.mx4_gemm(w, xs[k]), binding.mx4_gemm(w, *binding.mx4_quant(xs[k]))))
    torch.cuda.synchronize()
    for k in range(2):
        for a, b in got[k]:
            assert torch.equal(a, ref[k][0]) and torch.equal(b, ref[k][1])


def test_graphs_in_turn_on_one_workspace():
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    g = torch.Generator(device="cuda").manual_seed(6)
    w = [_random_tensor(640, 17408, g) for _ in range(2)]
    x = torch.randn(48, 17408, device="cuda", generator=g).half()
    need = binding.LIB.vq_mx4_workspace_bytes(640, 17408, 48)
    assert need > 0
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    ys, graphs = [], []
    for t in w:
        binding.mx4_gemm(t, x, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ys.append(binding.mx4_gemm(t, x, workspace=ws))
        graphs.append(graph)
    for k in range(4):
        x.copy_(torch.randn(48, 17408, device="cuda", generator=g).half())
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for t, y in zip(w, ys):
            assert torch.equal(y, binding.mx4_gemm(t, x))
        ws.fill_(0xff)


def test_refusals_on_the_gpu():
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    g = torch.Generator(device="cuda").manual_seed(7)
    w = _random_tensor(64, 256, g)
    x = torch.randn(6, 256, device="cuda").bfloat16()
    q, s = binding.mx4_quant(x)
    with pytest.raises(ValueError, match="contiguous"):
        binding.mx4_quant(torch.randn(6, 512, device="cuda")[:, :256])
    with pytest.raises(ValueError, match="contiguous"):
        binding.mx4_gemm(w, x.repeat(1, 2)[:, :256])
    with pytest.raises(ValueError, match="contiguous"):
        binding.mx4_gemm(w, q, s.repeat(1, 2)[:, :8])
    with pytest.raises(ValueError, match="contiguous"):
        binding.mx4_dequant(q.t().contiguous().t(), s)
    with pytest.raises(ValueError, match="y must"):
        binding.mx4_gemm(w, x, y=torch.empty(6, 63, device="cuda"))
    with pytest.raises(ValueError, match="y must be torch.float32"):
        binding.mx4_gemm(w, x, y=torch.empty(6, 64, dtype=torch.bfloat16, device="cuda"), y_dtype=torch.float32)
    with pytest.raises(ValueError, match="dtype"):
        binding.mx4_gemm(w, x, y=torch.empty(6, 64, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError, match="one tensor"):
        binding.mx4_gemm(binding.MX4Tensor(w.values.view(2, 32, 128), w.scales.view(2, 32, 8)), x)
    with pytest.raises(ValueError, match="cuda"):
        binding.mx4_gemm(w, x.cpu())
    off = torch.empty(6 * 256 + 4, device="cuda").bfloat16()[4:].view(6, 256)     # 8 bytes off
    with pytest.raises(binding.VQError, match="align"):
        binding.mx4_gemm(w, off)
    with pytest.raises(binding.VQError, match="align"):
        binding.mx4_quant(off)
    with pytest.raises(binding.VQError, match="workspace has"):
        need = binding.LIB.vq_mx4_workspace_bytes(64, 17408, 40)
        assert need > 0
        big = _random_tensor(64, 17408, g)
        binding.mx4_gemm(big, torch.zeros(40, 17408, device="cuda").half(),
                         workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    y = binding.mx4_gemm(w, x[:0])
    assert y.shape == (0, 64) and binding.mx4_quant(x[:0])[0].shape == (0, 128)


# ---- offsets past 32 bits -------------------------------------------------
# Scales of 1 and codes of at most 6 (16-bit x: whole numbers up to 4): sums of
# 8192 products are whole quarters below 2^20, exact in fp32 in any order, so the
# end of a large call equals a small one bit for bit.

def test_quantizer_past_4_gib():
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    T, C = (1 << 16) + 7, 33280                       # 2.18e9 values: 4.4 GB in fp16, 1.1 of codes
    x = torch.empty(T, C, dtype=torch.float16, device="cuda")
    x.view(torch.int16).fill_(0x3c00)
    x[-5:] = torch.randn(5, C, device="cuda").half()
    announce("mx4_quant past 4 GiB", T, C)
    q, s = binding.mx4_quant(x)
    sq, ss = binding.mx4_quant(x[-5:])
    assert torch.equal(q.view(torch.uint8)[-5:], sq.view(torch.uint8))
    assert torch.equal(s.view(torch.uint8)[-5:], ss.view(torch.uint8))
    assert torch.all(q.view(torch.uint8)[:-5] == 0x66).item()   # 1 = 4 * 2^-2
    binding.mx4_dequant(q, s, y=x)
    assert torch.equal(x[-5:], binding.mx4_dequant(sq, ss, dtype=torch.float16)) and torch.all(x[:-5] == 1).item()


@pytest.mark.parametrize("x", ["mx4", "bfloat16"])
def test_weight_past_4_gib(x):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    g = torch.Generator(device="cuda").manual_seed(8)
    R, C = (1 << 20) + 33, 8192
    w = _random_tensor(R, C, g, 127, 127)
    end = binding.MX4Tensor(w.values[-70:], w.scales[-70:])
    for T in (1, 40, 300):
        a = torch.randint(-4, 5, (T, C), device="cuda", generator=g).to(torch.bfloat16)
        a = (a,) if x != "mx4" else (torch.randint(0, 256, (T, C // 2), dtype=torch.uint8, device="cuda", generator=g),
                                     torch.full((T, C // 32), 127, dtype=torch.uint8, device="cuda"))
        announce("mx4_gemm weight past 4 GiB", x, T)
        y = binding.mx4_gemm(w, *a)
        assert torch.equal(y[:, -70:], binding.mx4_gemm(end, *a))
        assert y[:, :-70].abs().amax().item() > 0


@pytest.mark.parametrize("x,T,R,C", [("mx4", (1 << 20) + 9, 48, 8192), ("float16", (1 << 18) + 9, 48, 8192),
                                     ("mx4", (1 << 18) + 9, 5001, 256), ("bfloat16", (1 << 18) + 9, 5000, 256)])
def test_tokens_past_4_gib(x, T, R, C):
    """Activations, and outputs, of more than 4 GiB."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    g = torch.Generator(device="cuda").manual_seed(9)
    w = _random_tensor(R, C, g, 127, 127)
    if x == "mx4":
        a = (torch.randint(0, 256, (T, C // 2), dtype=torch.uint8, device="cuda", generator=g),
             torch.full((T, C // 32), 127, dtype=torch.uint8, device="cuda"))
    else:
        a = (torch.randint(-4, 5, (T, C), device="cuda", generator=g, dtype=torch.int8).to(_dt(x)),)
    announce("mx4_gemm tokens past 4 GiB", x, T, R, C)
    y = binding.mx4_gemm(w, *a)
    assert torch.equal(y[-130:], binding.mx4_gemm(w, *(t[-130:] for t in a)))
