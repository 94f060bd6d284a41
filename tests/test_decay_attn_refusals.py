"""Decayed linear attention: refusals of the arrays beside q, k, v (CPU; nothing is launched, the
addresses are never used)."""
import numpy as np
import pytest

import gated_delta_rule_63_b200 as G
from gated_delta_rule_63_b200 import build as B

D, GB = 128, 1 << 32
KEEP = np.array([0, 4000, 4096], np.int32)
TABLES = 0x10000      # log_decay, offsets and slots, 256 bytes apart
AT = dict(q=1 * GB, k=2 * GB, v=3 * GB, g=TABLES, cd=TABLES + 256, slot=TABLES + 512, h0=4 * GB, hT=5 * GB, pool=5 * GB,
          st=5 * GB, o=6 * GB, ws=7 * GB)


@pytest.fixture(scope="module")
def L():
    B.build()
    return G.lib()


def prefill(L, slots, **kw):
    a = {**AT, **kw}
    head = (a["q"], a["k"], a["v"], 0, 0, 0, a["g"], 1.0, 2, 4, a["cd"], KEEP.ctypes.data, 2)
    if slots:
        return L.gdr_decay_attn_prefill_slots(*head, a["pool"], 4, a["slot"], 1, a["o"], a["ws"], GB, None)
    return L.gdr_decay_attn_prefill(*head, a["h0"], a["hT"], a["o"], a["ws"], GB, None)


def decode(L, slots, **kw):
    a = {**AT, **kw}
    head = (a["q"], a["k"], a["v"], 0, 0, 0, a["g"], 1.0, 2, 4, a["st"])
    if slots:
        return L.gdr_decay_attn_decode_slots(*head, 4, a["slot"], a["o"], 3, None)
    return L.gdr_decay_attn_decode(*head, a["o"], 3, None)


def test_outputs_on_the_tables_are_refused(L):
    """log_decay, offsets or slots at the last bytes of an output, and an output from their last entry on."""
    need = int(L.gdr_decay_attn_prefill_workspace_size(KEEP.ctypes.data, 2, 4))
    assert need > 0
    n_state = 4 * D * D * 4
    for slots in (False, True):
        sizes = {"o": 4096 * 4 * D * 2, "ws": need, **({"pool": 4 * n_state} if slots else {"hT": 2 * n_state})}
        for name, size in sizes.items():
            for table in ("g", "cd", "slot") if slots else ("g", "cd"):
                assert prefill(L, slots, **{table: AT[name] + size - 4}) == 9, (slots, name, table)
                assert prefill(L, slots, **{table: AT[name]}) == 9, (slots, name, table)
        for name, size in {"o": 3 * 4 * D * 2, "st": (4 if slots else 3) * n_state}.items():
            for table in ("g", "slot") if slots else ("g",):
                assert decode(L, slots, **{table: AT[name] + size - 4}) == 9, (slots, name, table)
                assert decode(L, slots, **{table: AT[name] - 8}) == 9, (slots, name, table)


def test_tables_off_their_alignment_are_refused(L):
    """4-byte entries at an address that is not a multiple of 4: a load of them would fault."""
    for slots in (False, True):
        for by in (1, 2, 3):
            for table in ("g", "cd", "slot") if slots else ("g", "cd"):
                assert prefill(L, slots, **{table: AT[table] + by}) == 3, (slots, table)
            for table in ("g", "slot") if slots else ("g",):
                assert decode(L, slots, **{table: AT[table] + by}) == 3, (slots, table)
