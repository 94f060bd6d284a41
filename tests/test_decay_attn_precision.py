"""Decayed linear attention on a B200: the state has the error of fp32 sums, the returned one whatever
the tokens after a chunk are, and the one that o reads inside a prompt (e = 2^-23, an fp32 step).

One key per state row (keys e_0, e_1, ...): a chunk's product for a row is one value l^n v, held in
three bf16 terms, and nothing cancels.  Its error, relative to the value: the argument g n is
rounded once (|g n| e / 2 in the exponential), the exponential is good to 2 e, the product with v to
e / 2, the sum of its three terms to a step each: at most 6 e + |g n| e / 2.  Every later chunk or
piece multiplies by another exponential (2 e, and |g| 64 e / 2 from its argument) and adds (e / 2):
3 e.  Over a sequence of L tokens in c chunks: (6 + |g| L / 2 + 3 c) e of the magnitudes' sum.
Underflow adds what no relative bound covers: below 2^-126 an fp32 step is 2^-149, so each of those
6 + 3 c roundings is off by at most 2^-149, times |v| < 8 where it is the factor that is rounded;
and bf16's smallest step is 2^-133, below which a value's terms keep nothing: 2^-133 for each of the
tokens that write to a row.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_63_b200 as G
from oracle import oracle as O
from tests.test_decay_attn import CH, D, E, check, in_chunks, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    G.lib()
    yield
    assert G.get_device_error() == 0


@pytest.mark.parametrize("tail,decay", [(64, -0.5), (70, -0.3), (64, -1.0), (300, -0.06), (1700, -0.01)])
def test_state_of_a_sequence_that_ends_in_zero_keys(tail, decay):
    """64 ordinary tokens, then tokens that write nothing (a masked tail): the decayed sum of the
    first ones is all there is.  The longest one runs in segments."""
    q, k, v, cu, _ = make(51, [64 + tail], 1, 2)
    k[64:] = 0.0
    g = np.full(2, decay, np.float32)
    o, hT = run(q, k, v, g, cu)
    check(o, hT, q, k, v, g, cu, None, 1.0)


@pytest.mark.parametrize("tokens,tail,decay", [(128, 42, -0.5), (128, 102, -0.3), (40, 64, -1.0), (128, 300, -0.06),
                                               (128, 1722, -0.01), (128, 2300, -0.004), (700, 0, -0.004)])
def test_state_of_one_key_a_row(tokens, tail, decay):
    q, k, v, cu, _ = make(52, [tokens + tail], 1, 2)
    k[:] = 0.0
    at = np.arange(tokens)
    k[at, 0, at % D] = 1.0
    g = np.array([decay, 1.5 * decay], np.float32)
    _, hT = run(q, k, v, g, cu)
    _, ref = O.decay_attn(q, k, v, g, cu)
    _, size = O.decay_attn(q, k, np.abs(v), g, cu)
    L = int(cu[-1])
    bound = (6 + np.abs(g.astype(np.float64)) * L / 2 + 3 * ((L + CH - 1) // CH)) * E
    least = (6 + 3 * ((L + CH - 1) // CH)) * 8 * 2.0 ** -149 + (tokens // D + 1) * 2.0 ** -133
    assert np.abs(v).max() < 8
    err = np.abs(hT.double().cpu().numpy() - ref)[0]
    ok = bool(np.all(err <= bound[:, None, None] * size[0] + least))
    assert ok, float(np.max((err - least) / (E * size[0])))


@pytest.mark.parametrize("decay", [-0.02, -0.004, -0.002])
def test_o_is_not_too_small(decay):
    """A prompt in many segments: o against the oracle's rounded o, projected on the oracle's, which
    shows an error of one sign that the rounding to bf16 hides in each value.

    One sign can come from fp32 sums that are cut off instead of rounded, half a step in the mean:
    a value goes through four products of V' and K, eight of H and Q and four of V and P at full size
    (the others are of terms 2^-8 as large), and sum i of n weighs (i / n)^(1/2): 12 e / 2.
    Allowed are 16 e = 1.9e-6.  The rest is noise, the last bits that fall otherwise:
    2e-4 over the root of 8.4 million values, 7e-8."""
    T, hv = 8192, 8
    gen = torch.Generator(device="cuda").manual_seed(9)
    q, k, v = (torch.randn(T, hv, D, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
    g = torch.full((hv,), decay, device="cuda")
    cu = np.array([0, T], np.int32)
    assert G.decay_attn_workspace(cu, hv, "cuda") is not None
    o = G.decay_attn_prefill(q, k, v, g, torch.tensor(cu, device="cuda"), cu, scale=0.1)
    ref = in_chunks(q.double(), k.double(), v.double(), g.double(), cu, None, 0.1)[0]
    off = o.double() - ref.to(torch.bfloat16).double()
    shift = float((off * ref).sum() / (ref * ref).sum())
    assert abs(shift) <= 16 * E


@pytest.mark.parametrize("others", [0, 33])
def test_state_in_the_mean_over_a_head(others):
    """The returned state's error in the Frobenius norm, head by head, slow ones included; in segments, and
    (behind 33 short sequences) in one piece.

    Random values: the errors of a head's elements add as squares, and each source is relative to the
    state's own size.  Factors and products of V': 1.2 e.  A chunk's sums, should they be cut off: e / 2
    in the mean for four products at full size, 1.6 e.  The state's own two roundings a chunk, 0.41 e
    each time, over the 1 / (128 |g|) <= 16 chunks that it remembers: 1.6 e.  The decay of a chunk, good to
    e (1 - l^64) and |64 g| e / 2, of one sign, over the same memory: 0.75 e.  Together under 6 e = 7.2e-7;
    two terms of V' would leave 5e-6 to 1e-5."""
    q, k, v, cu, _ = make(53, [1] * others + [1500], 1, 5)
    g = np.array([-0.5, -0.06, -0.01, -0.004, -0.0005], np.float32)
    assert (G.decay_attn_workspace(cu, 5, "cuda") is not None) == (others == 0)
    _, hT = run(q, k, v, g, cu)
    _, ref = O.decay_attn(q, k, v, g, cu)
    err = hT[-1].double().cpu().numpy() - ref[-1]
    off = np.sqrt((err ** 2).sum((1, 2)) / (ref[-1] ** 2).sum((1, 2)))
    assert off.max() <= 6 * E, off


def test_state_of_the_smallest_values():
    """One chunk, one key a row, values from 2^-133 (bf16's least) to 2^-105: the bound of one product, and
    what lies below bf16's least step."""
    q, k, v, cu, _ = make(54, [64], 1, 2)
    k[:] = 0.0
    k[np.arange(64), 0, np.arange(64)] = 1.0
    v = O.round_bf16_f64(np.sign(v) * 2.0 ** np.random.default_rng(5).uniform(-133, -105, v.shape))
    g = np.array([0.0, -0.01], np.float32)
    _, hT = run(q, k, v, g, cu)
    _, ref = O.decay_attn(q, k, v, g, cu)
    err = np.abs(hT.double().cpu().numpy() - ref)
    bound = (6 + np.abs(g.astype(np.float64)) * 64 / 2)[None, :, None, None] * E * np.abs(ref) + 2.0 ** -133
    assert bool(np.all(err <= bound)), float(np.max(err / bound))
    assert bool(np.all(err[:, 0] == 0.0))                  # nothing decays: the values themselves
