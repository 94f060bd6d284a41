"""Decayed linear attention: the fp64 oracle's pins and the refusals (CPU), and the kernels
against the oracle on a B200.

Bounds, element by element (u = 2^-8, half a bf16 step; e = 2^-23, an fp32 step):
  o:  the result is rounded to bf16 once (u |o|); the products inside a chunk run on operands
      split into two bf16 values (u^2 of each product's size, A below), and every sum is fp32:
      at most 128 + 64 + 64 additions in turn, each off by a step of at most the sum of the
      magnitudes (B below): u |o| (1 + u) + 2 u^2 A + 256 e B.
      A = scale (l^(i+1) |q| |H| + sum_j l^(i-j) |q.k_j| |v_j|) with H at the chunk's start,
      B = scale |q| Habs, Habs the state with every product taken in magnitude.
  H:  the operands are split into three bf16 values (under an fp32 step), a chunk sums 64 of
      them in fp32, the decay factors are good to a few steps, and each chunk adds two
      roundings: (64 + 16 + 2 chunks) e Habs.
Decode: one fused multiply-add chain a value: 4 e Habs for H; o sums 128 of them.
"""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_63_b200 as G
from gated_delta_rule_63_b200 import build as B
from oracle import oracle as O

U, E = 2.0 ** -8, 2.0 ** -23
CH = 64                       # tokens of a chunk
D = 128


def make(seed, lengths, hk, hv, h0_std=None):
    """q, k, v as fp64 values of bf16 tensors, and an fp32 initial state."""
    rng = np.random.default_rng(seed)
    T = int(sum(lengths))
    q, k, v = (O.round_bf16_f64(rng.standard_normal((T, h, D))) for h in (hk, hk, hv))
    h0 = None if h0_std is None else (h0_std * rng.standard_normal((len(lengths), hv, D, D))).astype(np.float32)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    return q, k, v, cu, h0


def slopes(hv):
    return np.float32(-(2.0 ** (-8.0 * (np.arange(hv) + 1) / hv)))


def bounds(q, k, v, g, cu, h0, scale):
    """(A, B) for every o and Habs for every final state (see the module's text)."""
    hv = v.shape[1]
    key = np.arange(hv) // (hv // q.shape[1])
    lam = np.exp(np.asarray(g, np.float64))[:, None, None]
    A, Bo = np.zeros(v.shape), np.zeros(v.shape)
    Hs = np.zeros((len(cu) - 1, hv, D, D)) if h0 is None else np.array(h0, np.float64)
    Habs = np.abs(Hs)
    for i in range(len(cu) - 1):
        for t in range(int(cu[i]), int(cu[i + 1])):
            if (t - cu[i]) % CH == 0:
                Hc, part = np.abs(Hs[i]), []
            part.append((k[t, key], np.abs(v[t])))
            Hc = lam * Hc
            Hs[i] = lam * Hs[i] + k[t, key][:, :, None] * v[t][:, None, :]
            Habs[i] = lam * Habs[i] + np.abs(k[t, key])[:, :, None] * np.abs(v[t])[:, None, :]
            aq = np.abs(q[t, key])
            A[t] = np.einsum("hi,hij->hj", aq, Hc)
            for back, (kj, vj) in enumerate(reversed(part)):
                A[t] += (lam[:, 0] ** back if back else 1.0) * np.abs((q[t, key] * kj).sum(-1, keepdims=True)) * vj
            Bo[t] = np.einsum("hi,hij->hj", aq, Habs[i])
    return scale * A, scale * Bo, Habs


def in_chunks(q, k, v, g, cu, h0, scale):
    """The chunked form in fp64 (torch tensors, hk = hv): o, H and the A, B, Habs of the bounds."""
    n, hv = len(cu) - 1, v.shape[1]
    o, A, Bo = torch.zeros_like(v), torch.zeros_like(v), torch.zeros_like(v)
    H = torch.zeros(n, hv, D, D, dtype=v.dtype, device=v.device) if h0 is None else h0.clone()
    Habs = H.abs()
    for s in range(n):
        for a in range(int(cu[s]), int(cu[s + 1]), CH):
            b = min(a + CH, int(cu[s + 1]))
            x, y, z = (w[a:b].transpose(0, 1) for w in (q, k, v))          # [hv, m, D]
            i = torch.arange(b - a, device=v.device)
            low = (i[:, None] >= i).to(v.dtype)
            w = (g[:, None, None] * (i[:, None] - i).clamp(min=0)).exp() * low
            to_here = (g[:, None] * (i + 1)).exp()[..., None]
            to_end = (g[:, None] * (b - a - 1 - i)).exp()[..., None]
            P = x @ y.transpose(1, 2) * w
            o[a:b] = scale * (to_here * (x @ H[s]) + P @ z).transpose(0, 1)
            A[a:b] = scale * (to_here * (x.abs() @ H[s].abs()) + P.abs() @ z.abs()).transpose(0, 1)
            Bo[a:b] = scale * (to_here * (x.abs() @ Habs[s])
                               + (x.abs() @ y.abs().transpose(1, 2) * w) @ z.abs()).transpose(0, 1)
            last = (g * (b - a)).exp()[:, None, None]
            H[s] = last * H[s] + (y * to_end).transpose(1, 2) @ z
            Habs[s] = last * Habs[s] + (y.abs() * to_end).transpose(1, 2) @ z.abs()
    return o, H, A, Bo, Habs


def dev(x, dtype=torch.bfloat16):
    return torch.tensor(np.asarray(x, np.float64), dtype=torch.float64).to("cuda").to(dtype)


def packed(q, k, v, pad=0):
    """q, k, v as views of packed [q | k | v | pad] rows."""
    T, hk, hv = q.shape[0], q.shape[1], v.shape[1]
    rows = torch.full((T, (2 * hk + hv) * D + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    rows[:, : hk * D] = dev(q).view(T, -1)
    rows[:, hk * D: 2 * hk * D] = dev(k).view(T, -1)
    rows[:, 2 * hk * D: (2 * hk + hv) * D] = dev(v).view(T, -1)
    return (rows[:, : hk * D].unflatten(1, (hk, D)), rows[:, hk * D: 2 * hk * D].unflatten(1, (hk, D)),
            rows[:, 2 * hk * D: (2 * hk + hv) * D].unflatten(1, (hv, D)))


def check(o, hT, q, k, v, g, cu, h0, scale):
    ref_o, ref_h = O.decay_attn(q, k, v, g, cu, h0, scale)
    A, Bo, Habs = bounds(q, k, v, g, cu, h0, scale)
    got = o.double().cpu().numpy()[: int(cu[-1])]
    tol = U * np.abs(ref_o) * (1 + U) + 2 * U * U * A + 256 * E * Bo
    assert np.all(np.abs(got - ref_o) <= tol), float(np.max(np.abs(got - ref_o) / np.maximum(tol, 1e-300)))
    if hT is not None:
        n = (np.diff(cu) + CH - 1) // CH
        tol = ((64 + 16 + 2 * n) * E)[:, None, None, None] * Habs
        err = np.abs(hT.double().cpu().numpy() - ref_h)
        assert np.all(err <= tol), float(np.max(err / np.maximum(tol, 1e-300)))


# ---------------------------------------------------------------------------
# CPU: the oracle's pins
# ---------------------------------------------------------------------------

def test_oracle_written_out_by_hand():
    """d = 1: H = h0 l^t + sum l^(t-j) k_j v_j, o = scale q H."""
    q, k, v = np.array([[[2.0]], [[3.0]]]), np.array([[[5.0]], [[7.0]]]), np.array([[[11.0]], [[13.0]]])
    g = np.log(np.array([0.5]))
    o, H = O.decay_attn(q, k, v, g, [0, 2], np.array([[[[4.0]]]]), scale=0.25)
    h1 = 0.5 * 4 + 55
    h2 = 0.5 * h1 + 91
    assert np.allclose(o[:, 0, 0], [0.25 * 2 * h1, 0.25 * 3 * h2], rtol=1e-14) and np.isclose(H[0, 0, 0, 0], h2)


def test_oracle_equals_the_unrolled_sum():
    """o_t = scale sum_{j<=t} l^(t-j) (q_t.k_j) v_j + scale l^(t+1) H0^T q_t, heads grouped contiguously."""
    q, k, v, cu, h0 = make(1, [9], 2, 6, 0.5)
    g = slopes(6)
    o, H = O.decay_attn(q, k, v, g, cu, h0, 0.3)
    lam = np.exp(g.astype(np.float64))
    for h in range(6):
        w = np.tril(lam[h] ** (np.arange(9)[:, None] - np.arange(9)).clip(0))
        P = (q[:, h // 3] @ k[:, h // 3].T) * w
        inter = (lam[h] ** (np.arange(9) + 1))[:, None] * (q[:, h // 3] @ h0[0, h].astype(np.float64))
        assert np.allclose(o[:, h], 0.3 * (P @ v[:, h] + inter), rtol=1e-12, atol=1e-12)
        end = lam[h] ** 9 * h0[0, h].astype(np.float64) + (k[:, h // 3] * (lam[h] ** (8 - np.arange(9)))[:, None]).T @ v[:, h]
        assert np.allclose(H[0, h], end, rtol=1e-12, atol=1e-12)


def test_oracle_split_and_packed():
    """A sequence in two calls, the state handed over, is the sequence in one; packed is separate."""
    q, k, v, cu, h0 = make(2, [7, 5], 1, 2, 1.0)
    g = slopes(2)
    o, H = O.decay_attn(q, k, v, g, cu, h0)
    for n, (a, b) in enumerate([(0, 7), (7, 12)]):
        m = a + 3
        o1, H1 = O.decay_attn(q[a:m], k[a:m], v[a:m], g, [0, m - a], h0[n:n + 1])
        o2, H2 = O.decay_attn(q[m:b], k[m:b], v[m:b], g, [0, b - m], H1)
        assert np.array_equal(np.concatenate([o1, o2]), o[a:b]) and np.array_equal(H2[0], H[n])


def test_oracle_equals_the_chunked_form():
    """The chunked form in fp64, and the magnitudes of the bounds, on sequences around chunk borders."""
    q, k, v, cu, h0 = make(4, [130, 0, 64, 1], 2, 2, 1.0)
    g = np.array([-0.3, -1e-4])
    o, H = O.decay_attn(q, k, v, g, cu, h0, 0.7)
    A, Bo, Habs = bounds(q, k, v, g, cu, h0, 0.7)
    got = in_chunks(*(torch.tensor(x) for x in (q, k, v, g)), cu, torch.tensor(h0).double(), 0.7)
    for x, want in zip(got, (o, H, A, Bo, Habs)):
        assert np.allclose(x.numpy(), want, rtol=1e-10, atol=1e-10)


# ---------------------------------------------------------------------------
# CPU: refusals (nothing is launched; the addresses are never used)
# ---------------------------------------------------------------------------
P, GB = 0x10000, 1 << 32


@pytest.fixture(scope="module")
def L():
    B.build()
    return G.lib()


def cup(cu):
    a = np.asarray(cu, np.int32)
    return a, a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))


def test_prefill_refusals(L):
    keep, c = cup([0, 10, 15])

    def call(slots=False, **kw):
        a = dict(q=P, k=P + GB, v=P + 2 * GB, qs=0, ks=0, vs=0, g=P, scale=1.0, hk=2, hv=4, cd=P, ch=c, n=2, h0=None,
                 hT=P + 3 * GB, pool=P + 3 * GB, ns=4, slot=P, init=0, o=P + 4 * GB, ws=P + 5 * GB, wsb=GB)
        a.update(kw)
        head = [a[x] for x in ("q", "k", "v", "qs", "ks", "vs", "g", "scale", "hk", "hv", "cd", "ch", "n")]
        if slots:
            return L.gdr_decay_attn_prefill_slots(*head, *[a[x] for x in ("pool", "ns", "slot", "init", "o", "ws", "wsb")],
                                                  None)
        return L.gdr_decay_attn_prefill(*head, *[a[x] for x in ("h0", "hT", "o", "ws", "wsb")], None)
    for slots in (False, True):
        for name in ("q", "k", "v", "o", "g", "cd", "ch"):
            assert call(slots, **{name: None}) == 1, name
        for name in ("q", "k", "v", "o"):
            assert call(slots, **{name: P + 2}) == 3, name
        assert call(slots, hv=5) == 5 and call(slots, hk=1, hv=9) == 5
        assert call(slots, hk=0) == 2 and call(slots, hv=0) == 2 and call(slots, n=-1) == 2
        assert call(slots, qs=2 * D - 8) == 2 and call(slots, ks=2 * D - 8) == 2 and call(slots, vs=4 * D - 8) == 2
        assert call(slots, qs=2 * D + 4) == 3 and call(slots, ks=2 * D + 4) == 3 and call(slots, vs=4 * D + 4) == 3
        assert call(slots, ch=cup([0, 5, 3])[1]) == 4 and call(slots, ch=cup([1, 5, 6])[1]) == 4
        assert call(slots, o=P + 16) == 9                      # o on q
        assert call(slots, o=P + 2 * GB + (15 * 4 * D - 8) * 2) == 9   # o on the last values of v
        assert call(slots, o=P + 3 * GB + 64) == 9             # o on the states
        assert call(slots, n=0) == 0
    assert call(h0=P + 3 * GB + 64) == 9                       # h0 and hT partly overlap
    assert call(h0=P + 4 * GB) == 9                            # o on h0
    assert call(h0=P + 8) == 3 and call(hT=P + 8) == 3
    assert call(True, slot=None) == 1 and call(True, pool=None) == 1
    assert call(True, ns=-1) == 2 and call(True, init=2) == 2
    assert call(True, slot=P + 2) == 3 and call(True, pool=P + 8) == 3
    # nothing to do
    assert call(ch=cup([0, 0, 0])[1], hT=None, q=None, k=None, v=None, o=None, cd=None) == 0
    assert call(True, ch=cup([0, 0, 0])[1], ns=0, pool=None, q=None, k=None, v=None, o=None, cd=None) == 0


def test_prefill_refuses_bad_workspaces(L):
    """4096 tokens of four heads run in segments, whose states need a workspace."""
    keep, c = cup([0, 4096])
    need = L.gdr_decay_attn_prefill_workspace_size(c, 1, 4)
    assert need > 0 and need % (4 * D * D * 4) == 0
    assert L.gdr_decay_attn_prefill_workspace_size(cup([0, 200])[1], 1, 4) == 0
    call = lambda ws, nbytes, hT=P + 3 * GB: L.gdr_decay_attn_prefill(   # noqa: E731
        P, P + GB, P + 2 * GB, 0, 0, 0, P, 1.0, 2, 4, P, c, 1, None, hT, P + 4 * GB, ws, nbytes, None)
    assert call(None, need) == 6 and call(P + 5 * GB, need - 1) == 6 and call(P + 5 * GB + 8, need) == 3
    assert call(P + 4 * GB + 4096, need) == 9 and call(P + 2 * GB, need) == 9      # on o, on v
    assert call(P + 3 * GB - need + 16, need) == 9                                  # its end on hT


def test_decode_refusals(L):
    def call(slots=False, **kw):
        a = dict(q=P, k=P + GB, v=P + 2 * GB, qs=0, ks=0, vs=0, g=P, scale=1.0, hk=2, hv=4, st=P + 3 * GB, ns=4, slot=P,
                 o=P + 4 * GB, b=3)
        a.update(kw)
        head = [a[x] for x in ("q", "k", "v", "qs", "ks", "vs", "g", "scale", "hk", "hv", "st")]
        if slots:
            return L.gdr_decay_attn_decode_slots(*head, a["ns"], a["slot"], a["o"], a["b"], None)
        return L.gdr_decay_attn_decode(*head, a["o"], a["b"], None)
    for slots in (False, True):
        for name in ("q", "k", "v", "o", "g", "st"):
            assert call(slots, **{name: None}) == 1, name
        for name in ("q", "k", "v", "o", "st"):
            assert call(slots, **{name: P + 2}) == 3, name
        assert call(slots, hv=5) == 5 and call(slots, hk=0) == 2 and call(slots, b=-1) == 2
        assert call(slots, b=65536) == 2
        assert call(slots, qs=2 * D - 8) == 2 and call(slots, vs=4 * D + 4) == 3 and call(slots, ks=8) == 2
        assert call(slots, o=P + 3 * GB + 64) == 9 and call(slots, st=P) == 9 and call(slots, o=P) == 9
        assert call(slots, b=0, q=None) == 0
    assert call(True, slot=None) == 1 and call(True, ns=-1) == 2 and call(True, slot=P + 2) == 3


def test_workspace_size_of_bad_arguments(L):
    f = L.gdr_decay_attn_prefill_workspace_size
    assert f(None, 1, 4) == 0 and f(cup([0, 5])[1], 0, 4) == 0 and f(cup([0, 5])[1], 1, 0) == 0
    assert f(cup([0, 5, 4])[1], 2, 4) == 0


def test_binding_refuses_shapes():
    cpu = torch.zeros(4, 2, D, dtype=torch.bfloat16)
    with pytest.raises(ValueError):   # not on a GPU
        G.decay_attn_decode(cpu, cpu, cpu, torch.zeros(2), torch.zeros(4, 2, D, D))


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------

@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    G.lib()
    yield
    assert G.get_device_error() == 0


def run(q, k, v, g, cu, h0=None, scale=1.0, in_place=False, views=True, want_state=True, extra_rows=3):
    """The prefill over padded tensors: NaN rows behind the last sequence, canaries around o."""
    T = int(cu[-1])
    nan = lambda x: np.concatenate([x, np.full((extra_rows,) + x.shape[1:], np.nan)])   # noqa: E731
    qd, kd, vd = packed(nan(q), nan(k), nan(v), pad=8) if views else (dev(nan(q)), dev(nan(k)), dev(nan(v)))
    o = torch.full((T + extra_rows, v.shape[1], D), 7.0, dtype=torch.bfloat16, device="cuda")
    h0d = None if h0 is None else torch.tensor(h0, device="cuda")
    hT = None
    if want_state:
        hT = h0d if in_place else torch.full((len(cu) - 1, v.shape[1], D, D), float("nan"), device="cuda")
    G.decay_attn_prefill(qd, kd, vd, torch.tensor(np.asarray(g, np.float32), device="cuda"),
                         torch.tensor(cu, device="cuda"), cu, h0=h0d, hT=hT, o=o, scale=scale)
    torch.cuda.synchronize()
    assert bool((o[T:] == 7.0).all())                # rows behind the last sequence stay as they were
    if h0 is not None and not in_place:
        assert np.array_equal(h0d.cpu().numpy(), h0)
    return o, hT


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,hk,hv,h0_std,kind", [
    ([1], 1, 1, None, "slopes"),
    ([1], 1, 2, 1.0, "none"),
    ([2, 0, 1], 2, 2, 0.5, "slopes"),
    ([63], 1, 3, None, "slopes"),
    ([64], 2, 4, 1.0, "slopes"),
    ([65], 1, 2, 1.0, "fast"),
    ([128, 127, 129], 1, 2, 1.0, "slopes"),
    ([300], 2, 6, None, "none"),
    ([17, 0, 500, 1, 64, 200], 1, 8, 1.0, "slopes"),
    ([700], 3, 3, 0.3, "fast"),
    ([1500], 1, 1, 1.0, "slopes"),
    ([130, 1300, 1], 1, 2, 1.0, "grow"),
])
@pytest.mark.parametrize("views", [True, False])
def test_prefill_matches_oracle(gpu, lengths, hk, hv, h0_std, kind, views):
    q, k, v, cu, h0 = make(11 + len(lengths) + hv, lengths, hk, hv, h0_std)
    g = {"slopes": slopes(hv), "none": np.zeros(hv), "fast": -0.3 * 3.0 ** np.arange(hv),
         "grow": 1e-3 * (1 + np.arange(hv))}[kind].astype(np.float32)
    o, hT = run(q, k, v, g, cu, h0, scale=D ** -0.5, views=views)
    check(o, hT, q, k, v, g, cu, h0, D ** -0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("n_seqs", [33, 65, 90])
def test_prefill_of_many_sequences(gpu, n_seqs):
    """More sequences than are ever split, and more than ride in the launch parameters."""
    lengths = [int(x) for x in np.random.default_rng(n_seqs).integers(0, 70, n_seqs)]
    q, k, v, cu, h0 = make(12, lengths, 1, 1, 1.0)
    g = np.array([-0.02], np.float32)
    o, hT = run(q, k, v, g, cu, h0, scale=0.5)
    check(o, hT, q, k, v, g, cu, h0, 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,hv,h0_std", [([64 * 40], 48, None), ([64 * 37 + 5, 1, 0, 700], 16, 1.0),
                                               ([5000], 4, 1.0), ([9000, 100], 3, None)])
def test_prefill_in_segments(gpu, lengths, hv, h0_std):
    """Long sequences of few heads, which run as segments beside each other."""
    rng = np.random.default_rng(3)
    T, n = sum(lengths), len(lengths)
    t = lambda *s: torch.tensor(rng.standard_normal(s), device="cuda").to(torch.bfloat16)   # noqa: E731
    q, k, v = t(T, hv, D), t(T, hv, D), t(T, hv, D)
    g = torch.tensor(slopes(hv), device="cuda")
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    assert G.decay_attn_workspace(cu, hv, "cuda") is not None    # (split indeed)
    h0 = None if h0_std is None else torch.tensor(h0_std * rng.standard_normal((n, hv, D, D)), dtype=torch.float32,
                                                  device="cuda")
    ref_o, ref_h, A, Bo, Habs = in_chunks(q.double(), k.double(), v.double(), g.double(), cu,
                                          None if h0 is None else h0.double(), 0.1)
    hT = torch.empty(n, hv, D, D, device="cuda") if h0 is None else h0
    o = G.decay_attn_prefill(q, k, v, g, torch.tensor(cu, device="cuda"), cu, h0=h0, hT=hT, scale=0.1)
    assert bool(((o.double() - ref_o).abs() <= U * ref_o.abs() * (1 + U) + 2 * U * U * A + 256 * E * Bo).all())
    for i, x in enumerate(lengths):
        bound = (64 + 16 + 2 * ((x + CH - 1) // CH)) * E * Habs[i]
        assert bool(((hT[i].double() - ref_h[i]).abs() <= bound).all())


@pytest.mark.gpu
def test_prefill_heads_that_forget_at_once_and_slowly(gpu):
    """l = 0 (log_decay -inf), l below the smallest fp32, and l within 2^-24 of 1."""
    lengths = [200, 3]
    q, k, v, cu, h0 = make(31, lengths, 1, 4, 1.0)
    g = np.array([-np.inf, -120.0, -3e-8, -1e-5], np.float32)
    o, hT = run(q, k, v, g, cu, h0)
    check(o, hT, q, k, v, g, cu, h0, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", [[400, 70, 0, 1], [2600]])
def test_prefill_in_place_and_without_a_final_state(gpu, lengths):
    q, k, v, cu, h0 = make(32, lengths, 1, 2, 1.0)
    g = slopes(2)
    o1, h1 = run(q, k, v, g, cu, h0)
    o2, h2 = run(q, k, v, g, cu, h0, in_place=True)
    o3, _ = run(q, k, v, g, cu, h0, want_state=False)
    assert torch.equal(o1, o2) and torch.equal(o1, o3) and torch.equal(h1, h2)


@pytest.mark.gpu
def test_prefill_without_tokens_hands_the_states_on(gpu):
    q, k, v, cu, h0 = make(33, [0, 0], 1, 2, 1.0)
    _, hT = run(q, k, v, slopes(2), cu, h0)
    assert np.array_equal(hT.cpu().numpy(), h0)
    _, hT = run(q, k, v, slopes(2), cu)
    assert float(hT.abs().max()) == 0.0


@pytest.mark.gpu
def test_prefill_is_causal_where_values_are_not_finite(gpu):
    """NaN or infinity in a token's q, k or v: earlier tokens and other sequences keep their bits."""
    lengths = [150, 90]
    q, k, v, cu, h0 = make(34, lengths, 1, 2, 1.0)
    g = slopes(2)
    o, hT = run(q, k, v, g, cu, h0)
    for name, bad in (("q", np.nan), ("k", np.nan), ("v", np.nan), ("v", np.inf), ("k", -np.inf)):
        x = {"q": q.copy(), "k": k.copy(), "v": v.copy()}
        t = 100
        x[name][t, :, 5] = bad
        o2, h2 = run(x["q"], x["k"], x["v"], g, cu, h0)
        assert torch.equal(o[:t], o2[:t]), name
        assert torch.equal(o[150:240], o2[150:240]) and torch.equal(hT[1], h2[1]), name
        if name == "v":       # every later value of that column, and no other column
            assert not bool(torch.isfinite(o2[t:150, :, 5]).any())
            assert torch.equal(o[t:150, :, 6:], o2[t:150, :, 6:]) and torch.equal(o[t:150, :, :5], o2[t:150, :, :5])
            assert not bool(torch.isfinite(h2[0, :, :, 5]).any())
        elif name == "k":
            assert not bool(torch.isfinite(o2[t:150]).any())
        else:
            assert not bool(torch.isfinite(o2[t]).any()) and torch.equal(o[t + 1:150], o2[t + 1:150])
            assert torch.equal(hT[0], h2[0])


@pytest.mark.gpu
@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("lengths", [[70, 0, 5, 130], [0, 1900, 64, 1]])
def test_prefill_on_a_pool(gpu, init, lengths):
    """Entries in any order, a sequence without one, an empty sequence; other entries keep their
    bits; o and the states are those of the dense call."""
    q, k, v, cu, _ = make(35, lengths, 1, 2)
    g = slopes(2)
    pool = np.random.default_rng(5).standard_normal((6, 2, D, D)).astype(np.float32)
    slot = np.array([4, 2, 99, 0], np.int32)
    h0 = np.stack([pool[s] if init and s < 6 else np.zeros_like(pool[0]) for s in slot])
    pd = torch.tensor(pool, device="cuda")
    cu_d, gd = torch.tensor(cu, device="cuda"), torch.tensor(g, device="cuda")
    o = G.decay_attn_prefill_slots(dev(q), dev(k), dev(v), gd, cu_d, cu, pd, torch.tensor(slot, device="cuda"),
                                   init_from_pool=init)
    o2, hT = run(q, k, v, g, cu, h0, views=False)
    assert torch.equal(o, o2[: int(cu[-1])])
    for n, s in enumerate(slot):
        if s < 6:
            assert torch.equal(pd[s], hT[n])
    for e in (1, 3, 5):
        assert np.array_equal(pd[e].cpu().numpy(), pool[e])


@pytest.mark.gpu
def test_decode_matches_oracle_over_steps(gpu):
    """Steps on dense states against the oracle, and on a pool against the dense call bit for bit."""
    B_, hk, hv, steps = 5, 2, 6, 4
    q, k, v, cu, h0 = make(36, [steps] * B_, hk, hv, 1.0)
    g = np.array([-0.5, -0.01, -1e-6, 0.0, -np.inf, -30.0], np.float32)
    ref_o, ref_h = O.decay_attn(q, k, v, g, cu, h0, 0.5)
    _, Bo, Habs = bounds(q, k, v, g, cu, h0, 0.5)
    st, gd = torch.tensor(h0, device="cuda"), torch.tensor(g, device="cuda")
    pool = torch.full((9, hv, D, D), 3.0, device="cuda")
    slot = torch.tensor([7, 0, 3, 8, 1, -1, 9], dtype=torch.int32, device="cuda")   # the last two: padding rows
    pool[slot[:B_].long()] = st
    for t in range(steps):
        at = np.arange(B_) * steps + t
        o = G.decay_attn_decode(dev(q[at]), dev(k[at]), dev(v[at]), gd, st, scale=0.5)
        two = np.concatenate([at, at[:2]])
        qs, ks, vs = packed(q[two], k[two], v[two], pad=16)
        os = G.decay_attn_decode_slots(qs, ks, vs, gd, pool, slot, scale=0.5)
        assert torch.equal(os[:B_], o) and float(os[B_:].abs().max()) == 0.0
        err = np.abs(o.double().cpu().numpy() - ref_o[at])
        assert np.all(err <= U * np.abs(ref_o[at]) * (1 + U) + (128 + 4 * steps) * E * Bo[at])
    assert np.all(np.abs(st.double().cpu().numpy() - ref_h) <= 4 * steps * E * Habs)
    assert torch.equal(pool[slot[:B_].long()], st)
    for e in (2, 4, 5, 6):
        assert bool((pool[e] == 3.0).all())


@pytest.mark.gpu
def test_decode_of_an_empty_pool(gpu):
    q = torch.ones(2, 1, D, dtype=torch.bfloat16, device="cuda")
    o = torch.full((2, 1, D), 5.0, dtype=torch.bfloat16, device="cuda")
    G.decay_attn_decode_slots(q, q, q, torch.zeros(1, device="cuda"), torch.zeros(0, 1, D, D, device="cuda"),
                              torch.tensor([0, 1], dtype=torch.int32, device="cuda"), o=o)
    assert float(o.abs().max()) == 0.0


@pytest.mark.gpu
def test_prefill_then_decode_is_one_sequence(gpu):
    """A prompt prefilled in two calls and continued token by token is the whole sequence."""
    lengths = [333]
    q, k, v, cu, h0 = make(37, lengths, 1, 2, 1.0)
    g = slopes(2)
    pool = torch.zeros(3, 2, D, D, device="cuda")
    pool[1] = torch.tensor(h0[0], device="cuda")
    slot, gd = torch.tensor([1], dtype=torch.int32, device="cuda"), torch.tensor(g, device="cuda")
    parts = []
    for a, b in ((0, 100), (100, 330)):
        c = np.array([0, b - a], np.int32)
        parts.append(G.decay_attn_prefill_slots(dev(q[a:b]), dev(k[a:b]), dev(v[a:b]), gd,
                                                torch.tensor(c, device="cuda"), c, pool, slot, init_from_pool=True))
    for t in range(330, 333):
        parts.append(G.decay_attn_decode_slots(dev(q[t:t + 1]), dev(k[t:t + 1]), dev(v[t:t + 1]), gd, pool, slot))
    check(torch.cat(parts), pool[1:2], q, k, v, g, cu, h0, 1.0)


@pytest.mark.gpu
def test_calls_on_streams_and_in_graphs(gpu):
    """Two captured graphs with workspaces of their own, replayed on two streams at once, give the
    eager bits; so does a call on a side stream."""
    sets = []
    for seed, lengths in ((41, [2300, 65]), (42, [1700])):
        q, k, v, cu, h0 = make(seed, lengths, 1, 2, 1.0)
        s = dict(q=dev(q), k=dev(k), v=dev(v), log_decay=torch.tensor(slopes(2), device="cuda"),
                 cu_seqlens=torch.tensor(cu, device="cuda"), cu_seqlens_host=cu, h0=torch.tensor(h0, device="cuda"),
                 hT=torch.empty(len(lengths), 2, D, D, device="cuda"),
                 o=torch.empty(int(cu[-1]), 2, D, dtype=torch.bfloat16, device="cuda"),
                 workspace=G.decay_attn_workspace(cu, 2, "cuda"))
        G.decay_attn_prefill(**s)
        sets.append((s, s["o"].clone(), s["hT"].clone()))
    torch.cuda.synchronize()
    graphs = []
    for s, _, _ in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            G.decay_attn_prefill(**s)
        graphs.append(graph)
    side = [torch.cuda.Stream() for _ in sets]
    for s, _, _ in sets:
        s["o"].zero_()
        s["hT"].zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream in zip(graphs, side):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for s, o, hT in sets:
        assert torch.equal(s["o"], o) and torch.equal(s["hT"], hT)
        s["o"].zero_()
    torch.cuda.synchronize()
    G.decay_attn_prefill(**sets[0][0], stream=side[0])
    torch.cuda.synchronize()
    assert torch.equal(sets[0][0]["o"], sets[0][1])


@pytest.mark.gpu
def test_offsets_past_32_bits(gpu):
    """Rows 2^20 values apart and a pool of 140 000 entries: the last offsets are past 2^31 values.
    The same calls on dense copies and a small pool give the same bits."""
    T, wide, entries = 2200, 1 << 20, 140_000
    gen = torch.Generator(device="cuda").manual_seed(5)
    rows = torch.empty(T, wide, dtype=torch.bfloat16, device="cuda")
    for x in (rows[:, :D], rows[:, D:2 * D], rows[:, -D:]):
        x.copy_(torch.randn(T, D, generator=gen, device="cuda"))
    q, k, v = rows[:, None, :D], rows[:, None, D:2 * D], rows[:, None, -D:]
    g = torch.tensor([-0.01], device="cuda")
    pool = torch.empty(entries, 1, D, D, device="cuda")
    small = torch.randn(2, 1, D, D, generator=gen, device="cuda")
    pool[entries - 1] = small[1]
    cu = np.array([0, T], np.int32)
    cu_d = torch.tensor(cu, device="cuda")
    far, near = (torch.tensor([i], dtype=torch.int32, device="cuda") for i in (entries - 1, 1))
    o = G.decay_attn_prefill_slots(q, k, v, g, cu_d, cu, pool, far, init_from_pool=True)
    o2 = G.decay_attn_prefill_slots(*(x.contiguous() for x in (q, k, v)), g, cu_d, cu, small, near, init_from_pool=True)
    assert torch.equal(o, o2) and torch.equal(pool[entries - 1], small[1])
    # the last two rows as tokens of two sequences, the first of them a padding row
    far, near = (torch.tensor([-1, i], dtype=torch.int32, device="cuda") for i in (entries - 1, 1))
    o = G.decay_attn_decode_slots(q[-2:], k[-2:], v[-2:], g, pool, far)
    o2 = G.decay_attn_decode_slots(*(x[-2:].contiguous() for x in (q, k, v)), g, small, near)
    assert torch.equal(o, o2) and torch.equal(pool[entries - 1], small[1])


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu(gpu):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")   # noqa: E731
    cu = np.array([0, 4], np.int32)
    a = dict(q=z(4, 1, D), k=z(4, 1, D), v=z(4, 2, D), log_decay=z(2, dtype=torch.float32),
             cu_seqlens=torch.tensor(cu, device="cuda"), cu_seqlens_host=cu)
    for name, bad in (("q", z(1, 1, D).expand(4, 1, D)), ("q", z(4, 1, 64)), ("k", z(4, 2, D)), ("q", z(3, 1, D)), ("log_decay", z(1, dtype=torch.float32)),
                      ("h0", z(1, 1, D, D, dtype=torch.float32)), ("hT", z(2, 2, D, D, dtype=torch.float32)),
                      ("o", z(4, 1, D)), ("cu_seqlens", torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            G.decay_attn_prefill(**{**a, name: bad})
    for name, bad in (("q", z(4, 1, D, dtype=torch.float16)), ("log_decay", z(2)), ("h0", z(1, 2, D, D))):
        with pytest.raises(TypeError):
            G.decay_attn_prefill(**{**a, name: bad})
    with pytest.raises(G.GdrError) as e:      # o on v
        G.decay_attn_prefill(**a, o=a["v"])
    assert e.value.code == 9
