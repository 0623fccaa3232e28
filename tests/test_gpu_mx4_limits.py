"""The 4-bit operators at the ends of their ranges."""
import numpy as np
import pytest

from oracle import block_oracle as O
from tests.test_gpu_mx4_moe import Layer, _check

pytestmark = pytest.mark.gpu


def _weight(wq, ws):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    return binding.MX4Tensor(torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda())


@pytest.mark.parametrize("T", [1, 12, 70, 300])
def test_largest_scales(T):
    """Scale bytes 252 to 254.  Every value below 2^128 is taken exactly.  Those
    above are infinite to the reader, not finite beside 16-bit x, and as they are
    beside 4-bit x.  x is a power of two in one column: exact."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    C, R = 288, 3 * 16
    wq = np.zeros((R, C // 2), dtype=np.uint8)
    wq[:, 70] = np.tile(np.arange(16), 3)                        # column 140: every code under every scale
    ws = np.full((R, C // 32), 127, dtype=np.uint8)
    ws[:, 4] = np.repeat([252, 253, 254], 16)
    values = O.E2M1[np.tile(np.arange(16), 3)] * np.exp2(np.repeat([125.0, 126.0, 127.0], 16))
    held = np.where(np.abs(values) < 2.0 ** 128, values, np.copysign(np.inf, values))
    w = _weight(wq, ws)
    got = binding.mx4_dequant(w.values, w.scales, dtype=torch.float32).double().cpu().numpy()
    assert np.array_equal(got[:, 140], held)
    for dt in (torch.float16, torch.bfloat16):
        x = torch.zeros(T, C, dtype=dt, device="cuda")
        x[:, 140] = 2.0 ** -10
        y = binding.mx4_gemm(w, x).double().cpu().numpy()
        assert np.array_equal(y[:, np.isfinite(held)], np.tile(held[np.isfinite(held)] * 2.0 ** -10, (T, 1)))
        assert not np.isfinite(y[:, np.isinf(held)]).any()
    xq = np.zeros((T, C // 2), dtype=np.uint8)
    xq[:, 70] = 2                                               # 1.0
    xs = np.full((T, C // 32), 117, dtype=np.uint8)
    y = binding.mx4_gemm(w, torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda())
    assert np.array_equal(y.double().cpu().numpy(), np.tile(values * 2.0 ** -10, (T, 1)))


@pytest.mark.parametrize("T", [1, 9, 40])
def test_layer_largest_scales(T):
    """Down's weights under byte 252 are taken exactly; an expert with values of
    2^128 and above spoils the tokens that chose it, and no other."""
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    E, H, I = 3, 64, 32
    layer, r = Layer(E, H, I, ("limits",)), binding.Router(E, 1)
    layer.dn[1][1] = 252
    layer.tensors[1].scales[1] = 252
    l = torch.zeros(T, E, device="cuda")
    at = torch.arange(T, device="cuda") % 3
    l[torch.arange(T, device="cuda"), at] = 1.0
    x = (torch.randn(T, H, generator=torch.Generator().manual_seed(T)) * 2.0 ** -9).cuda().bfloat16()
    y = _check(layer, r, l, x)
    layer.tensors[1].scales[1, 2] = 254
    layer.tensors[1].values[1, 2] = 0x44                       # 2 * 2^127: row 2 of expert 1
    got, _, _ = binding.mx4_moe(r, *layer.tensors, l, x)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[at == 1, 2] = True
    assert torch.equal(got[~hit], y[~hit]) and not torch.isfinite(got[hit]).any()
