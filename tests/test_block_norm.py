"""The norms around a block: the fp64 oracle's pins and the refusals (CPU), and the kernel
against the oracle on a B200.

Bounds, element by element (u = 2^-8, half a bf16 step; e = 2^-23, an fp32 step):
  r:  the norm of x sums d squares in fp32 in a tree of at most 32 serial additions and 10
      levels, a square root and a division, then the weight, the gate, alpha and the sum:
      64 e (|residual| + |alpha gate u|), plus u |r| where r is rounded to bf16.
  y:  a sum of squares of r again: its relative error is at most twice r's over the row's rms,
      64 e on top; an error of r of its own; u |y| for the rounding to bf16.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_63_b200 as G
from gated_delta_rule_63_b200 import build as B
from oracle import oracle as O

U, E = 2.0 ** -8, 2.0 ** -23
P, GB = 0x10000, 1 << 32


# ---------------------------------------------------------------------------
# CPU
# ---------------------------------------------------------------------------

def test_oracle_written_out_by_hand():
    r, y = O.block_norm([[3.0, 4.0]], residual=[[1.0, 2.0]], gate=[2.0, 0.5], post_norm=True, w_post=[1.0, 10.0],
                        w_pre=[1.0, 3.0], alpha=0.1, eps_post=0.0, eps_pre=0.0)
    rms = np.sqrt(12.5)
    want = np.array([1 + 0.1 * 2 * 3 / rms, 2 + 0.1 * 0.5 * 10 * 4 / rms])
    assert np.allclose(r[0], want, rtol=1e-14)
    assert np.allclose(y[0], want / np.sqrt((want ** 2).mean()) * [1, 3], rtol=1e-14)


def test_oracle_equals_torch_rms_norm():
    rng = np.random.default_rng(0)
    x, res, w = rng.standard_normal((5, 24)), rng.standard_normal((5, 24)), rng.standard_normal(24)
    r, y = O.block_norm(x, residual=res, w_pre=w)
    assert np.array_equal(r, res + x)
    want = torch.nn.functional.rms_norm(torch.tensor(res + x), (24,), torch.tensor(w), 1e-6).numpy()
    assert np.allclose(y, want, rtol=1e-12)
    r, y = O.block_norm(x, post_norm=True)
    assert np.allclose(r, torch.nn.functional.rms_norm(torch.tensor(x), (24,), None, 1e-6).numpy(), rtol=1e-12)


def args(**kw):
    a = G.BlockNormArgs()
    base = dict(x=P, residual=P + GB, residual_out=P + 2 * GB, y=P + 3 * GB, alpha=1.0, eps_post=1e-6, eps_pre=1e-6)
    for name, value in {**base, **kw}.items():
        setattr(a, name, value)
    return a


def test_refusals():
    B.build()
    L = G.lib()

    def call(rows=4, d=64, **kw):
        import ctypes
        return L.gdr_block_norm(ctypes.byref(args(**kw)), rows, d, None)
    assert L.gdr_block_norm(None, 4, 64, None) == 1
    assert call(x=None) == 1 and call(residual_out=None, y=None) == 1
    assert call(rows=-1) == 2 and call(d=0) == 2 and call(d=60) == 2 and call(d=-8) == 2
    assert call(d=32776) == 5
    for name in ("x", "residual", "residual_out", "y", "gate", "w_post", "w_pre"):
        assert call(**{name: P + 5 * GB + 2}, post_norm=1) == 3, name
    for name in ("x_stride", "residual_stride", "residual_out_stride", "y_stride"):
        assert call(**{name: 56}) == 2 and call(**{name: 68}) == 3 and call(**{name: -64}) == 2, name
    assert call(gate=P + 5 * GB, gate_stride=56) == 2 and call(gate=P + 5 * GB, gate_stride=68) == 3
    assert call(post_norm=2) == 2 and call(residual_fp32=3) == 2 and call(gate_shared=-1) == 2
    assert call(eps_pre=-1.0) == 2 and call(eps_post=float("nan")) == 2
    assert call(w_post=P + 5 * GB) == 2                       # a weight without its norm
    assert call(w_pre=P + 5 * GB, y=None) == 2
    one = 64 * 2
    assert call(y=P + one) == 9                               # y on x, shifted
    assert call(y=P, y_stride=128) == 9                       # y on x, other rows
    assert call(y=P + GB) == 9                                # y on the residual
    assert call(y=P + 2 * GB) == 9                            # y on the new residual
    assert call(residual_out=P) == 9                          # the new residual on x
    assert call(residual_out=P + GB + one) == 9               # on the residual, shifted
    assert call(residual_out=P + GB, residual_stride=72) == 9 # in place with another stride
    assert call(gate=P + 3 * GB + 4 * one - 16, gate_shared=1) == 9   # y's last values are the gate
    assert call(w_pre=P + 2 * GB) == 9
    assert call(rows=0, x=None) == 0
    # rows side by side in one buffer meet only where their columns do
    side = dict(x_stride=256, y_stride=256)
    assert call(**side, x=P, y=P + one - 16) == 9 and call(**side, x=P + one, y=P + 16) == 9
    assert call(**side, x=P, y=P + 512 * 3 + one - 16) == 9       # the same, some rows on
    assert call(x=P, x_stride=256, y=P + one, y_stride=128) == 9  # with other strides they may


def test_binding_refuses_cpu_tensors():
    with pytest.raises(ValueError):
        G.block_norm(torch.zeros(2, 16, dtype=torch.bfloat16))


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


def make(seed, rows, d, wide, post, gate, with_res=True):
    rng = np.random.default_rng(seed)
    bf = lambda *s: O.round_bf16_f64(rng.standard_normal(s))                      # noqa: E731
    a = dict(x=bf(rows, d), residual=None, gate=None, post_norm=post, alpha=0.7)
    if with_res:
        a["residual"] = 3 * rng.standard_normal((rows, d)).astype(np.float32).astype(np.float64) if wide else bf(rows, d)
        a["residual"] = a["residual"].astype(np.float32).astype(np.float64)
    if gate:
        a["gate"] = bf(d) if gate == "channel" else bf(rows, d)
    a["w_post"] = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32) if post else None
    a["w_pre"] = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32)
    return a


def to_dev(a, wide):
    t = lambda x, dt: None if x is None else torch.tensor(np.asarray(x, np.float64)).to("cuda").to(dt)   # noqa: E731
    rdt = torch.float32 if wide else torch.bfloat16
    return {**a, "x": t(a["x"], torch.bfloat16), "residual": t(a["residual"], rdt), "gate": t(a["gate"], torch.bfloat16),
            "w_post": t(a["w_post"], torch.float32), "w_pre": t(a["w_pre"], torch.float32)}


def check(r, y, a, wide, eps=1e-6):
    ref_r, ref_y = O.block_norm(**a, eps_post=eps, eps_pre=eps)
    part = np.abs(ref_r - (0 if a["residual"] is None else a["residual"]))
    er = 64 * E * (part + (0 if a["residual"] is None else np.abs(a["residual"])))
    rms = np.sqrt((ref_r ** 2).mean(-1, keepdims=True) + eps)
    w = 1.0 if a["w_pre"] is None else np.abs(a["w_pre"].astype(np.float64))
    if r is not None:
        err = np.abs(r.double().cpu().numpy().reshape(ref_r.shape) - ref_r)
        assert np.all(err <= er + (0 if wide else U * np.abs(ref_r) * (1 + U)))
    if y is not None:
        rel = 64 * E + 2 * np.sqrt((er ** 2).mean(-1, keepdims=True)) / rms
        err = np.abs(y.double().cpu().numpy().reshape(ref_y.shape) - ref_y)
        assert np.all(err <= U * np.abs(ref_y) * (1 + U) + rel * np.abs(ref_y) + w * er / rms)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(1, 8), (3, 16), (1, 128), (7, 120), (5, 1000), (2, 1032), (1, 5120), (33, 5120),
                                    (300, 264), (4, 6144), (9, 8192), (2, 16392), (3, 32768)])
@pytest.mark.parametrize("wide,post,gate", [(False, False, None), (True, True, "channel"), (False, True, "row"),
                                            (True, False, "row"), (False, False, "channel")])
def test_matches_oracle(gpu, rows, d, wide, post, gate):
    a = make(rows * 7 + d, rows, d, wide, post, gate)
    r, y = G.block_norm(**to_dev(a, wide))
    assert r.dtype == (torch.float32 if wide else torch.bfloat16) and y.dtype == torch.bfloat16
    check(r, y, a, wide)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 5120])
def test_parts_left_out(gpu, d):
    """No residual, no weights, one output alone: the other's bits do not change."""
    a = make(3, 6, d, False, True, None)
    t = to_dev(a, False)
    r, y = G.block_norm(**t)
    r1, none = G.block_norm(**{**t, "w_pre": None}, want_y=False)
    assert none is None and torch.equal(r1, r)
    none, y1 = G.block_norm(**t, want_residual=False)
    assert none is None and torch.equal(y1, y)
    b = {**a, "residual": None, "w_post": None, "w_pre": None}
    check(*G.block_norm(**{**t, "residual": None, "w_post": None, "w_pre": None}), b, False)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
def test_in_place_and_strided_rows(gpu, wide):
    rows, d = 13, 1048
    a = make(4, rows, d, wide, True, "row")
    t = to_dev(a, wide)
    r, y = G.block_norm(**t)
    x2, res2 = t["x"].clone(), t["residual"].clone()
    r2, y2 = G.block_norm(**{**t, "x": x2, "residual": res2}, residual_out=res2, y=x2)
    assert r2 is res2 and y2 is x2 and torch.equal(r2, r) and torch.equal(y2, y)

    def spread(v, pad):
        buf = torch.full((rows, d + pad), float("nan"), dtype=v.dtype, device="cuda")
        buf[:, :d] = v
        return buf, buf[:, :d]
    (xb, xs), (rb, rs), (_, gs) = spread(t["x"], 8), spread(t["residual"], 24), spread(t["gate"], 40)
    r3, y3 = G.block_norm(**{**t, "x": xs, "residual": rs, "gate": gs}, residual_out=rs, y=xs)
    assert torch.equal(rs, r) and torch.equal(xs, y)
    assert bool(torch.isnan(xb[:, d:]).all()) and bool(torch.isnan(rb[:, d:]).all())


@pytest.mark.gpu
def test_offsets_past_32_bits(gpu):
    """Rows 2^20 values apart: the last ones lie past 2^31 values.  The bits of the dense call."""
    rows, d, wide = 2200, 640, 1 << 20
    t = to_dev(make(7, rows, d, False, True, "row"), False)
    buf = torch.empty(rows, wide, dtype=torch.bfloat16, device="cuda")
    parts = [buf[:, i * d:(i + 1) * d] for i in range(5)]
    for p, name in zip(parts, ("x", "residual", "gate")):
        p.copy_(t[name])
    r, y = G.block_norm(**t)
    G.block_norm(**{**t, "x": parts[0], "residual": parts[1], "gate": parts[2]}, residual_out=parts[1], y=parts[0])
    assert torch.equal(parts[1], r) and torch.equal(parts[0], y)


@pytest.mark.gpu
def test_rows_do_not_touch_each_other(gpu):
    """A row of NaN, one of infinities, one of zeros (eps 0: 0 / 0) leave the others' bits alone."""
    for d in (128, 5120):
        t = to_dev(make(5, 9, d, False, True, None), False)
        r, y = G.block_norm(**t, eps=0.0)
        x = t["x"].clone()
        x[2], x[4, 3], x[6] = float("nan"), float("inf"), 0.0
        r2, y2 = G.block_norm(**{**t, "x": x}, eps=0.0)
        for row in (0, 1, 3, 5, 7, 8):
            assert torch.equal(r[row], r2[row]) and torch.equal(y[row], y2[row])
        assert bool(torch.isnan(r2[2]).all()) and bool(torch.isnan(y2[2]).all())
        assert bool(torch.isnan(r2[6]).all())                  # 0 / sqrt(0 + 0)


@pytest.mark.gpu
def test_shapes_streams_and_graphs(gpu):
    a = make(6, 12, 640, False, False, None)
    t = to_dev(a, False)
    r, y = G.block_norm(**t)
    r3, y3 = G.block_norm(**{**t, "x": t["x"].view(3, 4, 640), "residual": t["residual"].view(3, 4, 640)})
    assert r3.shape == (3, 4, 640) and torch.equal(y3.view(12, 640), y) and torch.equal(r3.view(12, 640), r)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    r4, y4 = G.block_norm(**t, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(r4, r) and torch.equal(y4, y)
    ro, yo = torch.zeros_like(r), torch.zeros_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.block_norm(**t, residual_out=ro, y=yo)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ro, r) and torch.equal(yo, y)
    e, f = G.block_norm(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert e.shape == f.shape == (0, 64)


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu(gpu):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")   # noqa: E731
    x = z(4, 64)
    for kw in (dict(residual=z(3, 64)), dict(gate=z(4, 32)), dict(gate=z(32)), dict(w_pre=z(32, dtype=torch.float32)),
               dict(y=z(4, 72))):
        with pytest.raises(ValueError):
            G.block_norm(x, **kw)
    for kw in (dict(residual=z(4, 64, dtype=torch.float16)), dict(w_pre=z(64)), dict(y=z(4, 64, dtype=torch.float32)),
               dict(residual=z(4, 64, dtype=torch.float32), residual_out=z(4, 64))):
        with pytest.raises(TypeError):
            G.block_norm(x, **kw)
    with pytest.raises(G.GdrError) as e:
        G.block_norm(x, residual=z(4, 64), residual_out=x)
    assert e.value.code == 9
    with pytest.raises(G.GdrError) as e:
        G.block_norm(z(4, 60))
    assert e.value.code == 2
