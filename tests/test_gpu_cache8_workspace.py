"""One workspace for all calls of a program, the size of its largest (GPU): results are those with a workspace of each call's own."""
import numpy as np
import pytest
import torch

import gated_short_causal_amd as g
from test_cache8_workspace import DIRECT, plan
from test_gpu_cache8 import BF, DEV, I32, Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 32, 8), (128, 9, 3)])
def test_a_workspace_for_the_largest_call(D, Hq, Hkv):
    S, B, N, L, prefix, longest = 16, 16, 70, 2, 4096, 600
    npre, most = prefix // S, -(-longest // S)
    c = Cache("int8", npre + 4 * most, Hkv, S, D, B)
    # sequences may share pages: few are made
    table = torch.from_numpy(np.stack([npre + (i % 4) * most + np.arange(most) for i in range(N)]).astype(np.int32)).to(DEV)
    pages = torch.arange(npre, dtype=I32, device=DEV)
    lens = torch.tensor([(37 * i) % (longest - L) + L for i in range(N)], dtype=I32, device=DEV)
    q = torch.randn(N * L, Hq * D, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)

    def size(*call):
        return g.lfm2sc_attn_cached8_workspace_bytes(BF, D, Hq, Hkv, *call)

    largest = torch.full((size(N, L, prefix, longest) + 256,), 0xff, dtype=torch.uint8, device=DEV)
    whole = largest[:-256]
    for n, l, p, most_own in ((N, L, prefix, longest), (65, 1, prefix, longest), (64, 1, prefix, longest), (64, 1, prefix, 200), (3, 2, 4000, 100),
                              (1, 1, 1100, longest), (N, L, 0, longest), (17, 1, 0, 590), (1, 1, prefix, longest)):
        own = lens[:n].clamp(max=most_own)
        args = (q[:n * l], *c.args, pages, p, table[:n], own, l)
        a, b = (torch.full((n * l, Hq * D), float("nan"), dtype=BF, device=DEV) for _ in range(2))
        g.lfm2sc_attn_cached8(*args, a, whole, max_suffix_len=most_own)
        mine = torch.full((max(16, size(n, l, p, most_own)),), 0xff, dtype=torch.uint8, device=DEV)
        g.lfm2sc_attn_cached8(*args, b, mine, max_suffix_len=most_own)
        assert torch.equal(a, b) and torch.isfinite(a.float()).all(), (n, l, p, most_own)
    assert (largest[-256:] == 0xff).all()


def test_a_call_that_joins_nothing_takes_no_workspace():
    D, Hq, Hkv, S, N, own = 64, 8, 2, 16, 70, 1100
    most = -(-own // S)
    assert plan(D, Hq, Hkv, N, 1, 0, own).form == DIRECT and g.lfm2sc_attn_cached8_workspace_bytes(BF, D, Hq, Hkv, N, 1, 0, own) > 0
    c = Cache("e4m3", most, Hkv, S, D, 16)
    table = torch.arange(most, dtype=I32, device=DEV).expand(N, most).contiguous()
    lens = torch.full((N,), own, dtype=I32, device=DEV)
    q = torch.randn(N, Hq * D, device=DEV).to(BF)
    a, b = torch.empty_like(q), torch.empty_like(q)
    g.lfm2sc_attn_cached8(q, *c.args, None, 0, table, lens, 1, a, None, max_suffix_len=own)
    g.lfm2sc_attn_cached8(q, *c.args, None, 0, table, lens, 1, b, torch.empty(1 << 24, dtype=torch.uint8, device=DEV), max_suffix_len=own)
    assert torch.equal(a, b)
