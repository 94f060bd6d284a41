"""The block norm at the widths where its kernel changes (a warp a row up to 512 values, then 16, 32 and
64 values a thread), on a B200.  Bounds as in test_block_norm."""
import pytest
import torch

import gated_delta_rule_63_b200 as G
from tests.test_block_norm import check, make, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    G.lib()
    yield
    assert G.get_device_error() == 0


@pytest.mark.parametrize("rows,d", [(5, 248), (6, 256), (7, 264), (9, 504), (3, 512), (5, 520), (3, 8184), (2, 8200),
                                    (3, 12288), (1, 16376), (3, 16384)])
@pytest.mark.parametrize("wide,post,gate", [(False, False, None), (True, True, "channel"), (False, True, "row"),
                                            (True, False, "row"), (True, True, "row")])
def test_matches_oracle(rows, d, wide, post, gate):
    a = make(rows * 11 + d, rows, d, wide, post, gate)
    check(*G.block_norm(**to_dev(a, wide)), a, wide)


@pytest.mark.parametrize("d", [256, 512, 520, 8200, 16384, 32768])
def test_rows_in_one_buffer(d):
    """Padded rows in place: the bits of the dense call, and nothing written behind a row's end."""
    rows = 5
    t = to_dev(make(d, rows, d, False, True, "row"), False)
    r, y = G.block_norm(**t)
    buf = torch.full((rows, 3 * d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    x, res, gate = (buf[:, i * d:(i + 1) * d] for i in range(3))
    for part, name in ((x, "x"), (res, "residual"), (gate, "gate")):
        part.copy_(t[name])
    G.block_norm(**{**t, "x": x, "residual": res, "gate": gate}, residual_out=res, y=x)
    assert torch.equal(res, r) and torch.equal(x, y) and torch.equal(gate, t["gate"])
    assert bool((buf[:, 3 * d:] == 7.0).all())
