"""Decayed linear attention: a workspace that is made once for calls of any length."""
import numpy as np
import pytest
import torch

import gated_delta_rule_63_b200 as G
from gated_delta_rule_63_b200 import build as B

D = 128


@pytest.fixture(scope="module")
def L():
    B.build()
    return G.lib()


def size(L, lengths, hv):
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    return int(L.gdr_decay_attn_prefill_workspace_size(cu.ctypes.data, len(lengths), hv))


def test_a_longer_sequence_does_not_cover_a_shorter_one(L):
    """What a kept buffer has to reckon with: one sequence of 2432 tokens needs less than 2368."""
    assert size(L, [2432], 16) < size(L, [2368], 16)


@pytest.mark.parametrize("hv", [1, 2, 3, 4, 12, 16, 24, 48, 64, 148, 149, 296, 297])
def test_bound_covers_every_call(L, hv):
    rng = np.random.default_rng(hv)
    bound = L.gdr_decay_attn_prefill_workspace_bound
    for _ in range(400):
        n = int(rng.integers(1, 40))
        top = int(2 ** rng.uniform(4, 18))
        lengths = rng.integers(0, top + 1, n)
        lengths[rng.random(n) < 0.2] = 0
        need = size(L, lengths, hv)
        total = int(lengths.sum())
        assert need <= bound(total, n, hv)
        assert bound(total, n, hv) <= bound(total + int(rng.integers(0, 1000)), n + int(rng.integers(0, 3)), hv)


def test_bound_of_one_sequence_at_every_length(L):
    for hv in (1, 4, 16, 48):
        for T in range(1, 70000, 61):
            assert size(L, [T], hv) <= L.gdr_decay_attn_prefill_workspace_bound(T, 1, hv)


def test_bound_of_bad_arguments(L):
    f = L.gdr_decay_attn_prefill_workspace_bound
    assert f(-1, 1, 4) == 0 and f(10, 0, 4) == 0 and f(10, 1, 0) == 0 and f(1 << 31, 1, 4) == 0


@pytest.mark.gpu
def test_one_buffer_serves_all_lengths():
    """The same bits as with a workspace of the call's own, on a buffer of the bound."""
    hv = 4
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(5000, hv, D, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
    g = torch.tensor([-0.5, -0.1, -0.01, 0.0], device="cuda")
    ws = G.decay_attn_workspace_bound(5000, 2, hv, "cuda")
    for lengths in ([5000], [1700, 3300], [2368], [2432], [70]):
        cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        ends = [torch.empty(len(lengths), hv, D, D, device="cuda") for _ in range(2)]
        args = (q, k, v, g, torch.tensor(cu, device="cuda"), cu)
        a = G.decay_attn_prefill(*args, hT=ends[0], workspace=ws)
        b = G.decay_attn_prefill(*args, hT=ends[1])
        assert torch.equal(a[: cu[-1]], b[: cu[-1]]) and torch.equal(ends[0], ends[1])
    assert G.get_device_error() == 0
