"""More of the hybrid decoder's operators on the GPU against the fp64 oracle, and against formulas in 64 bits here."""
import numpy as np
import pytest
import torch

import gated_short_causal_amd as g
from oracle import hybrid as ho

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, I32 = torch.bfloat16, torch.int32


def _draft_calls(target, draft, tokens, ua, us):
    """Every sequence of the batch: whole numbers, equal to the oracle's."""
    N, L = tokens.shape
    V = target.shape[1]
    a, nxt = (torch.full((N,), -77, dtype=I32, device=DEV) for _ in range(2))
    ws = torch.full((g.lfm2sc_accept_drafts_workspace_bytes(N, L, V),), 255, dtype=torch.uint8, device=DEV)
    g.lfm2sc_accept_drafts(target.to(DEV), tokens.to(DEV), ua.to(DEV), us.to(DEV), a, nxt, ws, draft_probs=draft.to(DEV))
    wa, wn = ho.accept_drafts(target, tokens, ua, us, draft)
    assert (a.cpu().numpy() == wa).all(), (a, wa)
    assert (nxt.cpu().numpy() == wn).all(), (nxt, wn)


# the whole form with 1, 4 and 8 pieces in flight, the split form, rows shorter than a load
@pytest.mark.parametrize("V", [5, 700, 9001, 40003, 80003])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_drafts_entries_that_are_no_probabilities(V, dtype):
    """NaN and negative entries of the draft rows: nothing is taken from the target's weight, nothing added to it."""
    N, gen = 6, torch.Generator().manual_seed(V)
    target, draft = torch.rand(2 * N, V, generator=gen), torch.rand(N, V, generator=gen)
    draft[0, 1::3] = float("nan")
    draft[1, 1::2] = -draft[1, 1::2]
    draft[2, 1:] = -3.0                              # every weight would be 3 too large
    target[4, 2:] = -1.0                             # and the negative target entries would gain 2
    draft[3, 1:] = float("nan")
    target[6, : V // 2] = float("nan")               # NaN against NaN
    draft[4, 1:] = 2.0                               # nothing left but what is below
    draft[4, V - 1], target[8, V - 1] = -1.0, 0.0
    draft[5, 1:3], target[10, 1:3] = -1e-30, 0.0
    tokens = torch.zeros(N, 1, dtype=I32)
    draft[:, 0], target[::2, 0] = 1.0, 0.0           # token 0 is rejected
    target, draft = target.to(dtype), draft.to(dtype)
    for u in (0.0, 0.3, 0.77, 1 - 2 ** -24):
        _draft_calls(target, draft, tokens, torch.ones(N, 1), torch.full((N,), u))
