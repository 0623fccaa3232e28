"""The 4-bit operators' kernels over many steps of columns: every row of the
product's table forced, split and whole, with the planes that it leaves; every
kernel of the layer with columns that fill its ring more than once."""
import functools
import importlib.util
import os

import numpy as np
import pytest

from oracle import block_oracle as O
from tests.test_gpu_mx4 import _operands, _product_check
from tests.test_gpu_mx4_moe import _check, _inputs
from vq_dequant_matmul_gemv_amd import synth

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@functools.lru_cache(None)
def _table():
    spec = importlib.util.spec_from_file_location("mx4_plan_fit", os.path.join(ROOT, "profiles", "mx4_plan_fit.py"))
    fit = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fit)
    return fit.kernels()


# ---- product --------------------------------------------------------------

@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("kernel", range(24))
def test_every_kernel_over_many_steps(kernel, splits, monkeypatch):
    """145 blocks of columns: whole, and in exactly three splits whatever a
    kernel's splits are multiples of (52 to 64 blocks), the last one ending
    inside its unit; with four groups of waves its last groups have nothing.
    What is behind the planes, and a workspace that is not needed, stay as they
    are."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    C, k = 4640, _table()[kernel]
    part = -(-(-(-C // 32 // splits)) // k.unit) * k.unit
    assert -(-(C // 32) // part) == splits and C // 32 % part != 0 or splits == 1
    monkeypatch.setenv("VQMI_MX4_PLAN", f"{kernel},{splits}")
    for x in ("mx4",) if k.mx4 else ("float16", "bfloat16"):
        for T, R in ((3, 72), (37, 300), (270, 290)):
            ops = _operands(T, R, C, ("many steps", T, R), x)
            y = _product_check(ops)
            (xq, xs), (wq, ws) = ops
            w = binding.MX4Tensor(torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda())
            args = (xq.cuda(),) if xs is None else (torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda())
            used = splits * T * R if splits > 1 else 0
            need = max(binding.LIB.vq_mx4_workspace_bytes(R, C, T), 4 * used)
            assert binding.LIB.vq_mx4_workspace_bytes(R, C, T) >= 4 * used
            space = torch.full((need // 4 + 64,), -7.25e33, device="cuda")
            assert torch.equal(binding.mx4_gemm(w, *args, workspace=space), y)
            assert not torch.any(space[:used] == -7.25e33).item()
            assert torch.all(space[used:] == -7.25e33).item()


@pytest.mark.parametrize("kernel", range(12, 24))
def test_scales_fp16_cannot_hold_over_many_steps(kernel, monkeypatch):
    """With fp16 x, steps whose scales are fp16 values beside steps whose are not."""
    monkeypatch.setenv("VQMI_MX4_PLAN", f"{kernel},3")
    (xv, xs), (wq, ws) = _operands(37, 150, 4640, ("wide steps",), "float16", 100, 108)
    ws[:, 40:90] += 12
    ws[::7, 100:] += 40
    _product_check(((xv, xs), (wq, ws)))


# ---- layer ----------------------------------------------------------------

class _Experts:
    """A stack's values, an expert at a time."""
    def __init__(self, values, scales):
        self.shape = (values.shape[0], values.shape[1], 2 * values.shape[2])
        self.get = functools.lru_cache(None)(lambda e: O.mx4_values(values[e], scales[e]))

    def __getitem__(self, e):
        return self.get(int(e))


class _Layer:
    def __init__(self, E, H, I, lo=116, hi=124, shift=0):
        import torch
        from vq_dequant_matmul_gemv_amd import binding
        g = synth.rng("mx4-moe-steps", E, H, I)

        def stack(rows, cols):
            q = g.integers(0, 256, (E, rows, cols // 2), dtype=np.uint8)
            s = g.integers(lo, hi + 1, (E, rows, cols // 32), dtype=np.uint8)
            place = torch.zeros(s.size + 4, dtype=torch.uint8, device="cuda")[shift:shift + s.size].view(s.shape)
            place.copy_(torch.from_numpy(s))
            return _Experts(q, s), binding.MX4Tensor(torch.from_numpy(q).cuda(), place)

        self.E, self.H, self.I = E, H, I
        (self.gu, gu), (self.dn, dn) = stack(2 * I, H), stack(H, I)
        self.tensors = [gu, dn]

    def values(self):
        return self.gu, self.dn


def _eights(pairs, experts, inter):
    """Items of the gate and up products in groups of 8."""
    return (pairs + 7 * min(pairs, experts)) // 8 * (inter // 16)


@pytest.mark.parametrize("x", ["float16", "bfloat16"])
@pytest.mark.parametrize("T", [6, 40, 64])
def test_layer_groups_of_eight_and_grouped_down(T, x):
    """Gate and up by waves of their own with groups of 8 pairs (more than 5
    tokens, pairs >= experts, 1200 items and more): 5 steps of 256 columns; down
    by groups of 4: 4 steps, the next item's behind them."""
    from vq_dequant_matmul_gemv_amd import binding
    E, k, H, I = 33, 6, 1056, 1024
    assert T * k >= E and _eights(T * k, E, I) >= 1200
    _check(_Layer(E, H, I), binding.Router(E, k), *_inputs(T, E, H, ("eight", T), x), "bfloat16" if T == 40 else "float32")


@pytest.mark.parametrize("E,k,T", [(16, 4, 20), (64, 2, 20), (6, 2, 64), (5, 1, 6)])
def test_layer_groups_of_four(E, k, T):
    """More than 5 tokens with pairs < experts, or few items: gate and up by
    blocks whose four waves share 10 steps; down by groups of 4, 3 steps."""
    from vq_dequant_matmul_gemv_amd import binding
    H, I = 2336, 544
    assert T > 5 and (T * k < E or _eights(T * k, E, I) < 1200)
    _check(_Layer(E, H, I), binding.Router(E, k), *_inputs(T, E, H, ("four", E, T)))


@pytest.mark.parametrize("E,k,T", [(16, 4, 64), (8, 4, 64), (40, 4, 10)])
def test_layer_groups_of_eight_over_many_steps(E, k, T):
    """The same with 10 steps of a wave's own, down with 3."""
    from vq_dequant_matmul_gemv_amd import binding
    H, I = 2336, 544
    assert T * k >= E and _eights(T * k, E, I) >= 1200
    _check(_Layer(E, H, I), binding.Router(E, k), *_inputs(T, E, H, ("four", E, T)))


@pytest.mark.parametrize("T", [1, 2, 5])
@pytest.mark.parametrize("E,k,I", [(16, 4, 1312), (16, 4, 96), (256, 8, 32), (128, 6, 32), (40, 20, 320), (512, 8, 32)])
def test_layer_few_tokens(E, k, I, T):
    """Up to 5 tokens, routed by the layer's blocks (one shape of every number
    of experts a lane) or, with 20 slots and with 512 experts, by a launch
    before: 10 steps for four waves; down by each token's pairs (up to 20 slots
    for 8 waves) and by groups, 1 to 6 steps."""
    from vq_dequant_matmul_gemv_amd import binding
    H = 2336
    _check(_Layer(E, H, I), binding.Router(E, k), *_inputs(T, E, H, ("few", E, T)))


@pytest.mark.parametrize("T", [1, 4, 12, 64])
def test_layer_scales_fp16_cannot_hold_in_some_steps(T):
    from vq_dequant_matmul_gemv_amd import binding
    E, H, I = 33, 1056, 1024
    layer = _Layer(E, H, I, 100, 112)
    _check(layer, binding.Router(E, 6), *_inputs(T, E, H, ("wide", T), "float16"))


@pytest.mark.parametrize("T", [1, 4, 12, 64])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_layer_scales_off_their_words(T, shift):
    """Stacks of scales that start anywhere: the same bits."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    E, H, I = 33, 1056, 1024
    l, x = _inputs(T, E, H, ("off", T))
    r = binding.Router(E, 6)
    for a, b in zip(binding.mx4_moe(r, *_Layer(E, H, I).tensors, l, x),
                    binding.mx4_moe(r, *_Layer(E, H, I, shift=shift).tensors, l, x)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [4, 64])
def test_layer_over_many_steps_captured(T):
    """Replays of a layer of several steps, with eager work between them."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    E, H, I = 33, 1056, 1024
    layer, r = _Layer(E, H, I), binding.Router(E, 6)
    l, x = _inputs(T, E, H, ("captured", T))
    binding.mx4_moe(r, *layer.tensors, l, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.mx4_moe(r, *layer.tensors, l, x)
    for i in range(3):
        nl, nx = _inputs(T, E, H, ("captured", T, i))
        l.copy_(nl)
        x.copy_(nx)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, binding.mx4_moe(r, *layer.tensors, l, x)):
            assert torch.equal(a, b)
