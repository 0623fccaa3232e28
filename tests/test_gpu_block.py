"""The operators together, as a feed-forward block of a routed model runs them:
norm, router, routed VQ experts with their weights, a shared expert in e4m3,
and the norm behind the block with its gate and the residual.  Every step is
checked on the values that reached it; the whole block captured into a graph
gives the eager bits on new inputs."""
import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import vq_oracle as O
from tests.helpers import TOL, announce, row_rel_err, upload
from vq_dequant_matmul_gemv_amd import synth

pytestmark = pytest.mark.gpu

H, I, E, K = 512, 128, 16, 4          # hidden, expert intermediate, experts, slots


class Block:
    def __init__(self):
        import torch
        from vq_dequant_matmul_gemv_amd import binding
        self.b, self.torch = binding, torch
        self.gu_spec = synth.Spec(2 * I, H, 4, 8, 64, experts=E)
        self.dn_spec = synth.Spec(H, I, 4, 8, 64, experts=E)
        self.gu_arr, self.dn_arr = synth.tensor(self.gu_spec, "blk", "gu"), synth.tensor(self.dn_spec, "blk", "dn")
        self.gu, self.dn = upload(self.gu_arr, self.gu_spec), upload(self.dn_arr, self.dn_spec)
        g = synth.rng("blk", "rest")
        bf = lambda *s, scale=1.0, mean=0.0: torch.from_numpy(  # noqa: E731
            (mean + scale * g.normal(size=s)).astype(np.float32)).to(torch.bfloat16).cuda()
        self.pre, self.post = bf(H, scale=0.1, mean=1.0), bf(H, scale=0.1, mean=1.0)
        self.w_router = bf(E, H, scale=H ** -0.5)
        self.bias = torch.from_numpy((0.02 * g.normal(size=E)).astype(np.float32)).cuda()
        self.gate = bf(H)
        self.router = binding.Router(E, K, score="sigmoid", bias=self.bias, groups=4, top_groups=2,
                                     group_score="top2", scale=1.5)
        self.shared = {}
        for name, (r, c) in {"gu": (2 * I, H), "dn": (H, I)}.items():
            codes = B.e4m3_nearest(g.normal(size=(r, c)) * 60)
            scales = (0.02 * np.exp(0.2 * g.normal(size=(-(-r // 128), -(-c // 128)))) / 60).astype(np.float32)
            self.shared[name] = (codes, scales, binding.FP8Tensor(torch.from_numpy(codes).cuda(),
                                                                   torch.from_numpy(scales).cuda()))

    def run(self, x):
        b, torch = self.b, self.torch
        moe = b.moe_gemv if x.shape[0] <= 8 else b.moe_gemm
        s = {"x": x}
        _, s["h"], _ = b.norm(None, x, pre_weight=self.pre, store_residual=False)
        _, s["q"], s["qs"] = b.norm(None, x, pre_weight=self.pre, store_residual=False, h_dtype=torch.float8_e4m3fn)
        s["logits"] = (s["h"].float() @ self.w_router.float().t()).contiguous()
        s["ids"], s["rw"] = b.moe_route(self.router, s["logits"])
        s["act"] = moe(self.gu, s["h"], s["ids"], y_dtype=torch.bfloat16, epilogue="swiglu")
        s["routed"] = moe(self.dn, s["act"], s["ids"], x_per_slot=True, epilogue="combine", route_weights=s["rw"])
        s["sact"] = b.fp8_gemm(self.shared["gu"][2], s["q"], s["qs"], y_dtype=torch.bfloat16, epilogue="swiglu")
        s["sq"], s["sqs"] = b.fp8_quant(s["sact"])
        s["shared"] = b.fp8_gemm(self.shared["dn"][2], s["sq"], s["sqs"])
        s["out"] = s["routed"] + s["shared"]
        s["v"], s["next"], _ = b.norm(s["out"], x, post_weight=self.post, pre_weight=self.pre, gate=self.gate,
                                      gate_act="sigmoid", alpha=0.5)
        return s


@pytest.fixture(scope="module")
def block():
    return Block()


def _x(T, key):
    import torch
    return torch.from_numpy(synth.rng("blk-x", *key).normal(size=(T, H)).astype(np.float32)).to(torch.bfloat16).cuda()


def _f(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("T", [1, 5, 40, 130])
def test_block_step_by_step(block, T):
    import torch
    announce("block", T)
    s = block.run(_x(T, ("step", T)))
    torch.cuda.synchronize()
    # h: half a bf16 unit and 64 of fp32; its e4m3 twin half a step
    ref = B.norm(None, _f(s["x"]), pre_weight=_f(block.pre))["h"]
    assert np.all(np.abs(_f(s["h"]) - ref) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(ref))
    val = B.fp8_values(s["q"].view(torch.uint8).cpu().numpy(), s["qs"].cpu().numpy())
    sc = np.repeat(_f(s["qs"]), 128, axis=1)[:, :H]
    assert np.all(np.abs(val - ref) <= (1 + 2.0 ** -18) * np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * sc)
                  + 2.0 ** -18 * np.abs(ref))
    rid, rw = B.route(s["logits"].cpu().numpy(), K, score="sigmoid", bias=block.bias.cpu().numpy(), groups=4,
                      top_groups=2, group_score="top2", scale=1.5)
    ids = s["ids"].cpu().numpy()
    assert np.array_equal(ids, rid) and np.allclose(_f(s["rw"]), rw, rtol=2e-6, atol=0)
    # the routed experts on the ids and weights the router left
    a = block.gu_arr
    gu = O.moe_ref(a["codes"], a["codebook"], a["scales"], _f(s["h"]), ids, cols=H, d=4, log2_k=8, group=64,
                   x_per_slot=False)
    gate, up = gu[..., 0::2], gu[..., 1::2]
    act = gate / (1 + np.exp(-gate)) * up
    assert row_rel_err(_f(s["act"]).reshape(-1, I), act.reshape(-1, I)) <= 2.0 ** -8 + 4 * TOL
    a = block.dn_arr
    dn = O.moe_ref(a["codes"], a["codebook"], a["scales"], _f(s["act"]), ids, cols=I, d=4, log2_k=8, group=64,
                   x_per_slot=True)
    routed = (dn * _f(s["rw"])[..., None]).sum(axis=1)
    # errors of the slots add, the slots' sum may be smaller than they are
    assert np.abs(_f(s["routed"]) - routed).max() <= TOL * np.abs(dn * _f(s["rw"])[..., None]).sum(axis=1).max()
    # the shared expert
    u8 = lambda t: t.view(torch.uint8).cpu().numpy()  # noqa: E731
    y, _ = B.fp8_product(u8(s["q"]), s["qs"].cpu().numpy(), *block.shared["gu"][:2])
    y = y[:, 0::2] / (1 + np.exp(-y[:, 0::2])) * y[:, 1::2]
    assert np.abs(_f(s["sact"]) - y).max() <= 0.01 * np.abs(y).max()
    rq, rs = B.fp8_quant(_f(s["sact"]))
    assert np.array_equal(u8(s["sq"]), rq) and np.array_equal(s["sqs"].cpu().numpy(), rs)
    y, mag = B.fp8_product(rq, rs, *block.shared["dn"][:2])
    assert np.all(np.abs(_f(s["shared"]) - y) <= mag * 130 * 2.0 ** -23)
    n = B.norm(_f(s["out"]), _f(s["x"]), post_weight=_f(block.post), pre_weight=_f(block.pre), gate=_f(block.gate),
               gate_act="sigmoid", alpha=0.5)
    lim = 2.0 ** -8 * np.abs(n["v"]) + 64 * 2.0 ** -24 * (np.abs(n["u"]) + np.abs(n["r"]))
    assert np.all(np.abs(_f(s["v"]) - n["v"]) <= lim)
    assert np.all(np.abs(_f(s["next"]) - n["h"]) <= 2.0 ** -8 * np.abs(n["h"]) + 128 * 2.0 ** -24 * np.abs(n["h"]).max())


@pytest.mark.parametrize("T", [1, 40])
def test_block_captured_and_replayed(block, T):
    """The whole block in one graph; the combine adds slots atomically, so its
    last bits (and what follows) may differ: those are compared closely, the
    rest bit for bit."""
    import torch
    x = _x(T, ("cap", 0))
    block.run(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = block.run(x)
    for k in range(3):
        x.copy_(_x(T, ("cap", T, k)))
        graph.replay()
        torch.cuda.synchronize()
        e = block.run(x.clone())
        torch.cuda.synchronize()
        for name in ("h", "ids", "rw", "act", "sact", "sqs", "shared"):
            assert torch.equal(s[name], e[name]), name
        assert torch.equal(s["q"].view(torch.uint8), e["q"].view(torch.uint8))
        assert torch.allclose(s["routed"], e["routed"], rtol=0, atol=1e-5 * e["routed"].abs().max().item())
        assert torch.allclose(s["next"].float(), e["next"].float(), rtol=2.0 ** -7, atol=1e-3)


def test_two_streams_at_once(block):
    """Two blocks' calls on two streams, each with its own workspaces."""
    import torch
    xs = [_x(40, ("two", k)) for k in range(2)]
    ref = [block.run(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for st, x in zip(streams, xs):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append([block.run(x) for _ in range(3)][-1])
    torch.cuda.synchronize()
    for r, g in zip(ref, got):
        for name in ("h", "ids", "rw", "sact", "shared"):
            assert torch.equal(r[name], g[name]), name
