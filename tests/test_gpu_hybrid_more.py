"""More of the hybrid decoder's operators on the GPU against the fp64 oracle, and against formulas in 64 bits here."""
import numpy as np
import pytest
import torch

import gated_short_causal_amd as g
from oracle import hybrid as ho
from test_gpu_hybrid import _pages, _run_cached, _slack, _within

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


HALF = torch.finfo(BF).eps / 2
U = 2.0 ** -24                                       # half an fp32 step, relative


def _prompt64(q, k, v, cu, D, scale):
    """out and lse in 64 bits on the GPU, with the magnitudes that their errors scale with.

    An fp32 score is off by D sums of at most 2 U (rounded or cut) of scale sum |q||k|, by 3 U of its value from scale, log2 e
    and their product, by U of its value from the subtraction of the reference and by 2 U from exp2: terms(scale sum |q||k|)
    below.  lse takes these errors weighted with p; its sum of the exponentials adds one rounding per term of a tile of at
    most 64 keys and of a half's 32, and up to 4 per tile (sum, rescaling and its factor); the logarithm, the reference
    (within 16 of lse in base 2) and their sum add 8 U |lse| + 32 U.  out takes each p's error from its row's largest score
    terms, and the sum's error once more.
    """
    T, Hq, Hkv = q.shape[0], q.shape[1] // D, k.shape[1] // D
    q, k, v = q.double(), k.double(), v.double()
    out, spread = (torch.full((T, Hq * D), float("nan"), dtype=torch.float64, device=DEV) for _ in range(2))
    lse, lse_tol, p_tol = (torch.full((Hq, T), float("nan"), dtype=torch.float64, device=DEV) for _ in range(3))
    cu = cu.tolist()
    for a, b in zip(cu, cu[1:]):
        if a == b:
            continue
        future = torch.ones(b - a, b - a, dtype=torch.bool, device=DEV).triu(1)
        sums = 40 + 4 * (torch.arange(b - a, device=DEV) // 32 + 1)
        for h in range(Hq):
            c, kc = slice(h * D, h * D + D), slice(h // (Hq // Hkv) * D, h // (Hq // Hkv) * D + D)
            s = (scale * (q[a:b, c] @ k[a:b, kc].t())).masked_fill(future, float("-inf"))
            terms = (scale * (q[a:b, c].abs() @ k[a:b, kc].abs().t())).masked_fill(future, 0)
            p, z = torch.softmax(s, 1), torch.logsumexp(s, 1)
            out[a:b, c], spread[a:b, c], lse[h, a:b] = p @ v[a:b, kc], p @ v[a:b, kc].abs(), z
            lse_tol[h, a:b] = U * ((2 * D + 8) * (p * terms).sum(1) + 8 * z.abs() + 40 + sums)
            p_tol[h, a:b] = U * (2 * (2 * D + 8) * terms.amax(1) + 40 + sums)
    return out, spread, lse, lse_tol, p_tol.t().repeat_interleave(D, 1)


def _check_prompt(lens, Hq, Hkv, D, scale, amp=1.0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens)
    q = (torch.randn(T, Hq * D, generator=gen) * amp).to(BF).to(DEV)
    kv = torch.randn(T, 2 * Hkv * D, generator=gen).to(BF).to(DEV)
    k, v = kv[:, :Hkv * D], kv[:, Hkv * D:]
    cu = torch.tensor([0] + lens).cumsum(0).to(I32)
    out, lse = torch.full_like(q, float("nan")), torch.full((Hq, T), float("nan"), device=DEV)
    g.lfm2sc_attn_prefill(q, k, v, cu.to(DEV), D, out, lse=lse, scale=scale)
    want, spread, wlse, lse_tol, p_tol = _prompt64(q, k, v, cu, D, scale)
    off = (lse.double() - wlse).abs() / lse_tol
    assert (off <= 1).all(), ("lse", float(off.nan_to_num(9e9).max()))
    off = (out.double() - want).abs() / (HALF * (spread + want.abs()) + p_tol * spread)
    assert (off <= 1).all(), ("out", float(off.nan_to_num(9e9).max()))


@pytest.mark.parametrize("lens,Hq,Hkv,D", [([1], 8, 2, 128), ([2, 1, 3], 4, 1, 64), ([63], 2, 2, 64), ([65], 2, 1, 128), ([127, 1, 0, 128], 4, 2, 64),
                                           ([129, 31, 97], 6, 2, 128), ([300, 2], 12, 1, 64), ([33] * 90, 16, 8, 128), ([700], 9, 3, 128),
                                           ([1111], 2, 1, 64)])
@pytest.mark.parametrize("amp", [1.0, 30.0])
def test_prompt_lse_to_fp32(lens, Hq, Hkv, D, amp):
    """lse and out within what fp32 scores and sums leave; amp 30: scores of hundreds, most probabilities vanish."""
    _check_prompt(lens, Hq, Hkv, D, D ** -0.5, amp, seed=len(lens))


@pytest.mark.parametrize("T,Hq,Hkv,D", [(2100, 32, 8, 64), (4001, 32, 8, 64), (3333, 24, 8, 64), (5400, 12, 1, 64), (2051, 32, 4, 128),
                                        (3001, 32, 8, 128), (4500, 16, 2, 128)])
def test_prompt_one_sequence_of_many_row_blocks(T, Hq, Hkv, D):
    """One sequence whose workgroups are all resident: every other round of 256 / heads row blocks of 128 runs the other
    way, unless it is incomplete (2100, 3333, 5400, 2051 and 4500 tokens end in such a round)."""
    _check_prompt([T], Hq, Hkv, D, D ** -0.5, seed=T)


def _check_cached(lens, L, prefix, S, Hq, Hkv, D, most=None, seed=0):
    """Against the oracle; a page table of `most` pages a sequence, its unused entries no page numbers."""
    kv, pp, table = _pages(np.random.default_rng(seed), len(lens), lens, prefix, S, Hkv, D)
    if most is not None:
        wide = torch.full((len(lens), most), -1, dtype=I32)
        wide[:, 1::2] = 1 << 30
        wide[:, :table.shape[1]] = table
        for i, n in enumerate(lens):
            wide[i, -(-n // S):table.shape[1]] = -7
        table = wide
    q = torch.randn(len(lens) * L, Hq * D, generator=torch.Generator().manual_seed(seed)).to(BF)
    scale = D ** -0.5
    out = _run_cached(q, kv, pp, prefix, table, lens, L, D, scale, False)
    want, spread = ho.cached(q, kv[:, :, 0], kv[:, :, 1], pp, prefix, table.clamp(0, kv.shape[0] - 1), lens, L, scale)
    slack = _slack(q, torch.nan_to_num(kv.float()), D, scale)
    _within(out, want, HALF * (spread + np.abs(want)) + slack * spread, "out")


@pytest.mark.parametrize("lens,L,prefix,S,Hq,Hkv,D", [([37], 1, 500, 16, 32, 8, 64), ([5, 64, 200, 0], 1, 63, 16, 8, 2, 64), ([300, 1], 1, 0, 16, 4, 2, 128),
                                                      ([8, 9, 130], 8, 65, 64, 10, 2, 128), ([40] * 70, 1, 700, 32, 8, 2, 64)])
def test_cached_tables_wider_than_the_sequences(lens, L, prefix, S, Hq, Hkv, D):
    """A table of the longest context a server allows (32768 keys): most of its splits hold no key."""
    _check_cached(lens, L, prefix, S, Hq, Hkv, D, most=32768 // S)


@pytest.mark.parametrize("lens,L,prefix,S,Hq,Hkv,D", [([200, 150, 401], 150, 100, 16, 4, 2, 64), ([333], 333, 0, 32, 3, 1, 128), ([70, 600, 129], 129, 0, 16, 4, 4, 64),
                                                      ([140, 20, 0], 140, 1000, 64, 2, 1, 128)])
def test_cached_long_blocks(lens, L, prefix, S, Hq, Hkv, D):
    """Blocks of more tokens than a row block has rows; sequences shorter than the block."""
    _check_cached(lens, L, prefix, S, Hq, Hkv, D)
