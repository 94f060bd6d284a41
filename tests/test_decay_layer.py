"""A layer of decayed linear attention as it is served, on a B200: norm, projections, the
recurrence on a pool of states, gated norm, out-projection, the norms behind it, for new and
continued prompts and then token by token.

Every call's result is checked against the fp64 oracle of that call on the tensors it was given
(each within its own bounds), the whole step also as a CUDA graph.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_63_b200 as G
from oracle import oracle as O
from tests.test_block_norm import check as check_norm
from tests.test_decay_attn import E, U, check as check_attn
from tests.helpers import host_bits, ulp_diff_bf16

pytestmark = pytest.mark.gpu
D, HK, HV, HID = 128, 1, 3, 256
WIDTH = (2 * HK + 2 * HV) * D      # q | k | v | z


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    G.lib()
    yield
    assert G.get_device_error() == 0


class Layer:
    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        w = lambda *s: torch.tensor(rng.standard_normal(s) / np.sqrt(s[-1])).to("cuda").to(torch.bfloat16)   # noqa: E731
        f = lambda n: torch.tensor(1 + 0.1 * rng.standard_normal(n), dtype=torch.float32, device="cuda")     # noqa: E731
        self.w_in, self.w_out = w(WIDTH, HID), w(HID, HV * D)
        self.norm_w, self.w_pre, self.w_post, self.w_next = f(D), f(HID), f(HID), f(HID)
        self.gate = (0.5 * torch.tensor(rng.standard_normal(HID))).to("cuda").to(torch.bfloat16)
        self.log_decay = torch.tensor([-0.25, -0.02, -0.001], device="cuda")
        self.pool = torch.tensor(rng.standard_normal((5, HV, D, D)), dtype=torch.float32, device="cuda")

    def step(self, x, residual, recur):
        """One pass; recur(q, k, v) -> o is the recurrence.  Returns every tensor on the way."""
        r, h = G.block_norm(x, residual=residual, w_pre=self.w_pre)
        p = G.linear(h, self.w_in)
        T = p.shape[0]
        cut = lambda a, b: p[:, a * D: b * D].unflatten(1, (b - a, D))      # noqa: E731
        q, k, v = cut(0, HK), cut(HK, 2 * HK), cut(2 * HK, 2 * HK + HV)
        z = p[:, (2 * HK + HV) * D:].contiguous().view(T, HV, D)
        o = recur(q, k, v)
        y = G.gated_rmsnorm(o, z, self.norm_w)
        out = G.linear(y.view(T, HV * D), self.w_out)
        r2, nxt = G.block_norm(out, residual=r, post_norm=True, w_post=self.w_post, gate=self.gate, alpha=0.5,
                               w_pre=self.w_next)
        return dict(r=r, h=h, p=p, q=q, k=k, v=v, z=z, o=o, y=y, out=out, r2=r2, nxt=nxt)


def f64(t):
    return t.double().cpu().numpy()


def check_step(L, x, residual, s, cu, h0, states):
    check_norm(s["r"], s["h"], dict(x=f64(x), residual=f64(residual), gate=None, post_norm=False, w_post=None,
                                    w_pre=L.w_pre.cpu().numpy(), alpha=1.0), False)
    check_attn(s["o"], states, f64(s["q"]), f64(s["k"]), f64(s["v"]), L.log_decay.cpu().numpy(), cu, h0, D ** -0.5)
    # gated norm: at most one bf16 step from the rounded oracle; projections: half a step and fp32 sums
    ref = O.round_bf16(O.gated_rmsnorm(f64(s["o"]), f64(s["z"]), L.norm_w.cpu().numpy()))
    assert int(ulp_diff_bf16(host_bits(s["y"]), ref).max()) <= 1
    for a, w, got in ((f64(s["h"]), f64(L.w_in), s["p"]), (f64(s["y"]).reshape(len(x), -1), f64(L.w_out), s["out"])):
        exact, size = a @ w.T, np.abs(a) @ np.abs(w).T
        assert np.all(np.abs(f64(got) - exact) <= U * np.abs(exact) * (1 + U) + a.shape[1] * E * size)
    check_norm(s["r2"], s["nxt"], dict(x=f64(s["out"]), residual=f64(s["r"]), gate=f64(L.gate), post_norm=True,
                                       w_post=L.w_post.cpu().numpy(), w_pre=L.w_next.cpu().numpy(), alpha=0.5), False)


def inputs(rng, T):
    t = lambda: torch.tensor(rng.standard_normal((T, HID))).to("cuda").to(torch.bfloat16)   # noqa: E731
    return t(), t()


def test_prompts_then_tokens_on_one_pool():
    rng = np.random.default_rng(1)
    L = Layer(2)
    pool0 = L.pool.clone()
    # two prompts into entries 3 and 0 (continued from what is there), one into none
    lengths = [70, 130, 5]
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    cu_d = torch.tensor(cu, device="cuda")
    slot = torch.tensor([3, 0, -1], dtype=torch.int32, device="cuda")
    x, res = inputs(rng, int(cu[-1]))
    s = L.step(x, res, lambda q, k, v: G.decay_attn_prefill_slots(q, k, v, L.log_decay, cu_d, cu, L.pool, slot,
                                                                  init_from_pool=True, scale=D ** -0.5))
    h0 = np.stack([pool0[3].cpu().numpy(), pool0[0].cpu().numpy(), np.zeros((HV, D, D), np.float32)])
    check_step(L, x, res, {**s}, cu, h0, None)
    _, ends = O.decay_attn(f64(s["q"]), f64(s["k"]), f64(s["v"]), L.log_decay.cpu().numpy(), cu, h0)
    for e in (1, 2, 4):
        assert torch.equal(L.pool[e], pool0[e])
    assert np.allclose(L.pool[3].cpu().numpy(), ends[0], rtol=1e-4, atol=1e-4 * np.abs(ends[0]).max())
    # then tokens for both, with a padding row, from the same entries
    for _ in range(3):
        before = L.pool.cpu().numpy()
        dslot = torch.tensor([0, -1, 3], dtype=torch.int32, device="cuda")
        x, res = inputs(rng, 3)
        s = L.step(x, res, lambda q, k, v: G.decay_attn_decode_slots(q, k, v, L.log_decay, L.pool, dslot,
                                                                     scale=D ** -0.5))
        assert float(s["o"][1].abs().max()) == 0.0
        live = {k: (t[[0, 2]] if k in ("q", "k", "v", "o") else t) for k, t in s.items()}
        check_attn(live["o"], L.pool[[0, 3]], f64(live["q"]), f64(live["k"]), f64(live["v"]),
                   L.log_decay.cpu().numpy(), np.array([0, 1, 2], np.int32), before[[0, 3]], D ** -0.5)


def test_the_step_replays_from_a_graph():
    rng = np.random.default_rng(3)
    L = Layer(4)
    lengths = [300, 64, 1]
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    cu_d = torch.tensor(cu, device="cuda")
    slot = torch.tensor([1, 4, 2], dtype=torch.int32, device="cuda")
    x, res = inputs(rng, int(cu[-1]))
    pool0 = L.pool.clone()

    def recur(q, k, v):
        return G.decay_attn_prefill_slots(q, k, v, L.log_decay, cu_d, cu, L.pool, slot, scale=D ** -0.5)
    eager = L.step(x, res, recur)
    after = L.pool.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = L.step(x, res, recur)
    L.pool.copy_(pool0)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for name in ("o", "out", "r2", "nxt"):
        assert torch.equal(s[name], eager[name]), name
    assert torch.equal(L.pool, after)
