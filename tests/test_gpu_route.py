"""vq_moe_route against a plain loop in 64 bits: the ids exactly, the weights
to fp32 rounding, over scores, biases, groups, types, odd sizes and masks."""
import numpy as np
import pytest

from oracle import block_oracle as O
from tests.helpers import announce
from vq_dequant_matmul_gemv_amd import synth

pytestmark = pytest.mark.gpu

# Weights are exp, sums of at most 64 terms and one quotient in at least 32
# bits: an exp of a rounded argument x (|x| e^x <= 0.37 of the largest, times
# 2^-24) and its own 2 units, 6 tree additions, the quotient, the scale and the
# final rounding stay below 32 half units of the row's largest weight.
REL = 32 * 2.0 ** -24


def _logits(T, E, dtype, key, masked=False):
    import torch
    g = synth.rng("route-logits", *key)
    x = (1.5 * g.normal(size=(T, E)) + g.normal(size=E)).astype(np.float32)
    t = torch.from_numpy(x).to(dtype)
    if masked:
        t[:, torch.from_numpy(g.random(E) < 0.2)] = torch.finfo(dtype).min
        t[torch.from_numpy(g.random((T, E)) < 0.15)] = -np.inf
        t[torch.from_numpy(g.random((T, E)) < 0.02)] = np.nan
        t[torch.from_numpy(g.random((T, E)) < 0.01)] = np.inf
        t[torch.from_numpy(g.random(T) < 0.2)] = -np.inf          # padded tokens
        t[0] = -np.inf
    return t


def _check(logits, top_k, bias=None, **kw):
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    T, E = logits.shape
    announce("moe_route", tuple(logits.shape), str(logits.dtype), top_k, "bias" if bias is not None else "", kw)
    r = binding.Router(E, top_k, bias=None if bias is None else bias.cuda(), **kw)
    # poisoned outputs with a guard behind the last row
    ids = torch.full(((T + 1) * top_k,), 777, dtype=torch.int32, device="cuda")
    w = torch.full(((T + 1) * top_k,), 777.0, device="cuda")
    n = T * top_k
    got = binding.moe_route(r, logits.cuda(), ids=ids[:n].view(T, top_k), weights=w[:n].view(T, top_k))
    torch.cuda.synchronize()
    rid, rw = O.route(logits.float().numpy(), top_k, bias=None if bias is None else bias.numpy(), **kw)
    assert np.array_equal(got[0].cpu().numpy(), rid)
    gw = got[1].cpu().numpy().astype(np.float64)
    top = np.abs(rw).max(axis=1, keepdims=True)
    assert np.all(np.abs(gw - rw) <= REL * top + 1e-37), np.max(np.abs(gw - rw))
    assert torch.all(ids[n:] == 777).item() and torch.all(w[n:] == 777.0).item()


def _dt(name):
    import torch
    return getattr(torch, name)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("E,k,T", [(1, 1, 5), (2, 1, 1), (7, 7, 13), (64, 6, 65), (65, 8, 3), (128, 64, 9),
                                   (160, 6, 31), (256, 8, 130), (500, 10, 17), (1024, 16, 6)])
def test_plain_choice(score, dtype, E, k, T):
    _check(_logits(T, E, _dt(dtype), ("plain", score, E, T)), k, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k,groups,top_groups,group_score,bias", [
    (256, 8, 8, 4, "top2", True), (256, 8, 8, 4, "top2", False), (256, 8, 8, 3, "max", True),
    (160, 6, 8, 3, "max", False), (96, 4, 3, 2, "top2", True), (72, 12, 72 // 2, 20, "top2", True),
    (64, 8, 64, 40, "max", True), (64, 3, 64, 3, "top2", False), (1000, 20, 10, 5, "top2", True),
    (256, 32, 1, 1, "max", True), (6, 2, 2, 1, "top2", True),
])
def test_groups_and_bias(score, renorm, E, k, groups, top_groups, group_score, bias):
    import torch
    g = synth.rng("route-bias", E, groups)
    b = torch.from_numpy((0.05 * g.normal(size=E)).astype(np.float32)) if bias else None
    x = _logits(67, E, torch.float32, ("groups", E, groups))
    _check(x, k, b, score=score, groups=groups, top_groups=top_groups, group_score=group_score,
           renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("groups,top_groups,group_score,bias", [
    (1, 1, "max", False), (1, 1, "max", True), (8, 3, "max", False), (8, 3, "top2", False), (8, 3, "top2", True)])
def test_masks(score, dtype, groups, top_groups, group_score, bias):
    """-inf, NaN, +inf and lowest-value logits, rows with nothing left, a bias
    with -inf and NaN in it."""
    import torch
    b = None
    if bias:
        g = synth.rng("route-mask-bias")
        b = torch.from_numpy((0.05 * g.normal(size=96)).astype(np.float32))
        b[5], b[17], b[80] = -np.inf, np.nan, np.inf
    _check(_logits(83, 96, _dt(dtype), ("mask", dtype), masked=True), 8, b, score=score, groups=groups,
           top_groups=top_groups, group_score=group_score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_ties_go_to_the_lowest(score, bias):
    """Rows of equal values, of few values, of +0 and -0, of one value a group."""
    import torch
    E = 96
    g = synth.rng("route-ties")
    rows = [np.zeros(E), np.where(g.random(E) < 0.5, 0.0, -0.0), g.integers(0, 3, E), np.repeat(np.arange(8), 12),
            np.full(E, -100.0), np.full(E, 50.0), np.full(E, np.finfo(np.float32).min)]
    x = torch.from_numpy(np.stack(rows).astype(np.float32))
    b = torch.from_numpy(g.integers(0, 2, E).astype(np.float32)) if bias else None
    for kw in (dict(), dict(groups=8, top_groups=3, group_score="top2"), dict(groups=8, top_groups=3)):
        _check(x, 10, b, score=score, **kw)


def test_nearly_equal_keys_are_ordered_in_64_bits():
    """Sigmoid scores a few 32-bit units apart behind a bias: the order of the
    64-bit keys decides, expert by expert and group by group."""
    import torch
    E, T = 256, 40
    g = synth.rng("route-near")
    base = g.normal(size=(T, 1))
    x = (base + 2.0 ** -22 * g.integers(-8, 9, size=(T, E))).astype(np.float32)
    b = torch.from_numpy((0.25 + 2.0 ** -24 * g.integers(-4, 5, size=E)).astype(np.float32))
    for score in ("sigmoid", "softmax"):
        _check(torch.from_numpy(x), 8, b, score=score)
        _check(torch.from_numpy(x), 8, b, score=score, groups=8, top_groups=4, group_score="top2")
        _check(torch.from_numpy(x), 8, None, score=score, groups=8, top_groups=4, group_score="top2")


@pytest.mark.parametrize("low", [-80.0, -300.0, -700.0])
def test_far_negative_scores_keep_their_weights(low):
    """Sigmoids far below fp32's range still renormalise to their ratios."""
    import torch
    x = torch.tensor([[low, low + 1.0, low + 2.0, low - 1.0]])
    _check(x, 3, score="sigmoid")
    _check(x, 3, score="softmax")


def test_empty_batch_and_other_stream_and_capture():
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    r = binding.Router(64, 4)
    ids, w = binding.moe_route(r, torch.zeros(0, 64, device="cuda"))
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    x = _logits(33, 64, torch.float32, ("stream",)).cuda()
    ref = binding.moe_route(r, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = binding.moe_route(r, x, stream=s)
    s.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    # a captured call replays on new logits
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gi, gw = binding.moe_route(r, buf)
    for seed in range(3):
        buf.copy_(_logits(33, 64, torch.float32, ("replay", seed)))
        graph.replay()
        torch.cuda.synchronize()
        ri, rw = binding.moe_route(r, buf)
        assert torch.equal(gi, ri) and torch.equal(gw, rw)


# ---- keys close to each other, and sums that cancel ------------------------

@pytest.mark.parametrize("E,k,T", [(64, 6, 33), (160, 16, 21), (256, 8, 40), (256, 32, 9), (512, 64, 5), (20, 20, 7)])
@pytest.mark.parametrize("cluster", [2, 3, 9])
def test_clusters_of_close_keys(E, k, T, cluster):
    """Sigmoid scores plus a bias in clusters of neighbours far closer than an
    fp32 score's error, exact ties among them: at the edge of the chosen and
    inside, with clusters that fit the chosen and the next one and that do not."""
    import torch
    g = synth.rng("route-cluster", E, k, cluster)
    n = -(-E // cluster)
    x = np.repeat(g.normal(size=(T, n)), cluster, axis=1)[:, :E].astype(np.float32)
    x = np.nextafter(x, np.where(g.random((T, E)) < 0.5, np.float32(9), np.float32(-9)).astype(np.float32))
    b = np.zeros(E, dtype=np.float32)
    b[g.random(E) < 0.1] = np.float32(2.0 ** -30)
    order = g.permutation(E)
    _check(torch.from_numpy(np.ascontiguousarray(x[:, order])), k, torch.from_numpy(b), score="sigmoid")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("big", [10.0, 200.0, 1000.0, 3e6, 3e38])
def test_group_sums_that_cancel(score, big):
    """Two experts of a group with biases of nearly opposite size: the group's
    sum is small, its keys' rounding errors are not."""
    import torch
    E, groups, T = 64, 16, 1200
    g = synth.rng("route-cancel", score, str(big))
    b = np.full(E, -big, dtype=np.float32)
    b[0::4] = big
    b[1::4] = -big
    b[2::4] = -big * 1.5 if big < 1e38 else -big
    x = torch.from_numpy((0.01 * g.normal(size=(T, E))).astype(np.float32))
    _check(x, 5, torch.from_numpy(b), score=score, groups=groups, top_groups=5, group_score="top2")


@pytest.mark.parametrize("T", [8191, 8192, 8195])
@pytest.mark.parametrize("kw", [dict(), dict(score="sigmoid", groups=8, top_groups=3, group_score="top2")])
def test_many_tokens(T, kw):
    """Both sides of the token count at which a token takes fewer lanes."""
    import torch
    g = synth.rng("route-many", T)
    x = _logits(T, 144, torch.bfloat16, ("many", T), masked=True)
    b = torch.from_numpy((0.05 * g.normal(size=144)).astype(np.float32)) if kw else None
    _check(x, 6, b, **kw)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("score,bias", [("sigmoid", True), ("softmax", True), ("softmax", False)])
def test_many_tokens_with_groups_of_whole_lanes(dtype, score, bias):
    import torch
    g = synth.rng("route-many-whole", dtype)
    x = _logits(8209, 256, _dt(dtype), ("many-whole", dtype), masked=True)
    b = torch.from_numpy((0.05 * g.normal(size=256)).astype(np.float32)) if bias else None
    _check(x, 8, b, score=score, groups=8, top_groups=4, group_score="top2", scale=2.5)
    _check(x, 16, b, score=score, groups=16, top_groups=5, renormalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,T", [(8, 2, 3), (96, 8, 21), (32, 8, 8200), (256, 8, 9), (120, 12, 5)])
def test_groups_masked_by_the_lowest_bias(score, E, groups, T):
    """A bias of fp32's lowest value on whole groups: their two best sum to
    below every fp32 number, and they stay in play behind the others."""
    import torch
    g = synth.rng("route-lowest", E, groups)
    size = E // groups
    low = torch.finfo(torch.float32).min
    b = torch.from_numpy((0.05 * g.normal(size=E)).astype(np.float32))
    b[size:2 * size] = low                     # one whole group
    b[(groups - 1) * size:] = 0.75 * low       # another, a little less low
    if groups > 4:
        b[2 * size + 1:3 * size] = low         # one with a single ordinary expert
    x = torch.from_numpy((1.5 * g.normal(size=(T, E))).astype(np.float32))
    if T > 8191:                               # many tokens: four a wave; the groups behind the first two are low
        b[2 * size:] = low
        return _check(x, 2 * size + 6, b, score=score, groups=groups, top_groups=groups - 1, group_score="top2")
    for top_groups in (groups, groups - 1):
        k = min(64, top_groups * size)
        for gs in ("top2", "max"):
            _check(x, k, b, score=score, groups=groups, top_groups=top_groups, group_score=gs)


def test_a_slot_count_out_of_range_allocates_nothing():
    import torch
    from vq_dequant_matmul_gemv_amd import binding
    x = torch.zeros(4096, 64, device="cuda")
    binding.moe_route(binding.Router(64, 8), x)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    for k in (65, 1 << 20, 1 << 30, 0, -1):
        with pytest.raises(binding.VQError, match="top_k"):
            binding.moe_route(binding.Router(64, k), x)
    assert torch.cuda.max_memory_allocated() - before <= 1 << 20
