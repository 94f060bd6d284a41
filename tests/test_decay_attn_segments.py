"""Decayed linear attention in segments: values that are not finite, heads that forget at once, and
the numbers of sequences at which the launch changes (32: the most that are split, 64: the most whose
offsets ride in the launch parameters).  Bounds as in test_decay_attn."""
import numpy as np
import pytest
import torch

import gated_delta_rule_63_b200 as G
from tests.test_decay_attn import D, check, make, run, slopes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    G.lib()
    yield
    assert G.get_device_error() == 0


@pytest.mark.parametrize("name,bad", [("q", np.nan), ("q", np.inf), ("k", np.nan), ("k", -np.inf), ("v", np.nan),
                                      ("v", np.inf)])
def test_causal_where_values_are_not_finite(name, bad):
    """One value in any piece of any segment: earlier tokens and the other sequence keep their bits."""
    T, other = 1900, 90
    q, k, v, cu, h0 = make(61, [T, other], 1, 2, 1.0)
    g = slopes(2)
    assert G.decay_attn_workspace(cu, 2, "cuda") is not None
    o, hT = run(q, k, v, g, cu, h0)
    for t in (0, 70, 200, 290, 330, 640, 1000, 1300, 1860, T - 1):
        x = {"q": q.copy(), "k": k.copy(), "v": v.copy()}
        x[name][t, :, 5] = bad
        o2, h2 = run(x["q"], x["k"], x["v"], g, cu, h0)
        assert torch.equal(o[:t], o2[:t]), t
        assert torch.equal(o[T:T + other], o2[T:T + other]) and torch.equal(hT[1], h2[1]), t
        if name == "v":
            assert not bool(torch.isfinite(o2[t:T, :, 5]).any()), t
            for cols in (slice(0, 5), slice(6, D)):
                assert torch.equal(o[t:T, :, cols], o2[t:T, :, cols]), t
                assert torch.equal(hT[0, :, :, cols], h2[0, :, :, cols]), t
            assert not bool(torch.isfinite(h2[0, :, :, 5]).any()), t
        elif name == "k":
            assert not bool(torch.isfinite(o2[t:T]).any()), t
            assert not bool(torch.isfinite(h2[0, :, 5]).any()), t
            assert torch.equal(hT[0, :, :5], h2[0, :, :5]) and torch.equal(hT[0, :, 6:], h2[0, :, 6:]), t
        else:
            assert not bool(torch.isfinite(o2[t]).any()), t
            assert torch.equal(o[t + 1:T], o2[t + 1:T]) and torch.equal(hT, h2), t


def test_initial_state_that_is_not_finite():
    """A NaN in the initial state: every output of its column, and no other sequence's."""
    q, k, v, cu, h0 = make(62, [1700, 65], 1, 2, 1.0)
    g = slopes(2)
    o, hT = run(q, k, v, g, cu, h0)
    h0[0, 1, 7, 9] = np.nan
    o2, h2 = run(q, k, v, g, cu, h0, in_place=True)
    assert not bool(torch.isfinite(o2[:1700, 1, 9]).any()) and not bool(torch.isfinite(h2[0, 1, 7, 9]))
    o2[:1700, 1, 9] = o[:1700, 1, 9]
    h2[0, 1, 7, 9] = hT[0, 1, 7, 9]
    assert torch.equal(o[:1765], o2[:1765]) and torch.equal(hT, h2)


def test_heads_that_forget_at_once_and_slowly():
    q, k, v, cu, h0 = make(63, [1600, 3], 1, 4, 1.0)
    g = np.array([-np.inf, -120.0, -3e-8, -1e-5], np.float32)
    assert G.decay_attn_workspace(cu, 4, "cuda") is not None
    o, hT = run(q, k, v, g, cu, h0)
    check(o, hT, q, k, v, g, cu, h0, 1.0)


@pytest.mark.parametrize("n_seqs,longest", [(32, 60), (32, 1500), (33, 1500), (64, 130), (65, 130)])
def test_numbers_of_sequences_at_the_limits(n_seqs, longest):
    rng = np.random.default_rng(n_seqs)
    lengths = [int(x) for x in rng.integers(0, 40, n_seqs)]
    lengths[n_seqs // 3] = longest
    q, k, v, cu, h0 = make(64, lengths, 1, 1, 1.0)
    g = np.array([-0.02], np.float32)
    assert (G.decay_attn_workspace(cu, 1, "cuda") is not None) == (n_seqs <= 32 and longest > 1000)
    o, hT = run(q, k, v, g, cu, h0, scale=0.5)
    check(o, hT, q, k, v, g, cu, h0, 0.5)
