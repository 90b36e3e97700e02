"""LFM2SC_CHECK=1 looks at the device data that a call uses, and at no more (GPU; the switch is read once per process, hence
a child).  Status 6 is LFM2SC_ERR_PRECONDITION."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_COMMON = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
import gated_short_causal_amd as g
I32, BF, d = torch.int32, torch.bfloat16, "cuda"

def status(call):
    try:
        call()
        return 0
    except g.Lfm2scError as e:
        return e.status

def ints(*v):
    return torch.tensor(v, dtype=I32, device=d)

"""

_PAGES = _COMMON + """
pool = torch.randn(8, 16, 2, 64, device=d).to(BF)
q, out = torch.randn(3, 128, device=d).to(BF), torch.empty(3, 128, dtype=BF, device=d)
ws = torch.empty(1 << 20, dtype=torch.uint8, device=d)
def cached(table, lens):
    return status(lambda: g.lfm2sc_attn_cached(q, pool, pool, ints(1), 10, table, lens, 1, out, ws))
wild = 1 << 30
table = ints(2, 3, 7, 4, -1, wild, -1, -1, -1).reshape(3, 3)   # 33..48, 1..16 and 0 keys are in use
s = [cached(table, ints(48, 16, 0)), cached(table, ints(33, 1, 0)), cached(table, ints(33, 17, 0)), cached(table, ints(33, 16, 1)),
     cached(table, ints(49, 16, 0)), cached(table, ints(33, -1, 0)), cached(table[:1].contiguous(), ints(48)), cached(table[:2].contiguous(), ints(48, 48))]
torch.cuda.synchronize()
print("STATUS", s)
"""

_TOKENS = _COMMON + """
p, u = torch.rand(9, 50, device=d), torch.rand(3, 2, device=d)
r = torch.empty(2, 3, dtype=I32, device=d)
ws = torch.empty(1 << 12, dtype=torch.uint8, device=d)
def drafts(tokens, n):
    return status(lambda: g.lfm2sc_accept_drafts(p, tokens, u, u.reshape(-1)[:3].contiguous(), r[0], r[1], ws, num_drafts=n))
tokens = ints(0, 49, 7, -1, 50, 1 << 30).reshape(3, 2)         # two, one and no drafts are in use
s = [drafts(tokens, ints(2, 1, 0)), drafts(tokens, ints(1, 1, 0)), drafts(tokens, ints(2, 2, 0)), drafts(tokens, ints(2, 1, 1)),
     drafts(tokens, None), drafts(tokens, ints(2, 1, -1))]
torch.cuda.synchronize()
print("STATUS", s)
"""


@pytest.mark.parametrize("script,want", [(_PAGES, [0, 0, 6, 6, 6, 6, 0, 6]), (_TOKENS, [0, 0, 6, 6, 6, 6])], ids=["pages", "tokens"])
def test_entries_past_a_sequences_length_are_not_checked(script, want):
    r = subprocess.run([sys.executable, "-c", script, ROOT], env=dict(os.environ, LFM2SC_CHECK="1"), capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    line = [x for x in r.stdout.splitlines() if x.startswith("STATUS")][0]
    assert line == f"STATUS {want}", line
