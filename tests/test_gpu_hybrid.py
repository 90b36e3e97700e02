"""The hybrid decoder's operators on the GPU against the fp64 oracle.

Tolerances, derived from the roundings (HALF = half a bf16 step, relative):
  attention   each p is rounded once before the product with v, the output once: HALF * (sum p |v| + |out|);
  gradients   p, ds and out (in delta = d_out.out) are rounded once, the gradient once: the oracle's bounds + HALF |g|;
  lse         fp32 sums of D products and of the exponentials;
  everything  fp32 scores: D products summed in fp32 move a score by at most D 2^-24 sum |q||k|, hence every p by that
              much relatively: SLACK of the same magnitudes, with 2^-20 for a score's size of up to 16 D / 2.
Drafts' outputs are whole numbers and have to be equal.
"""
import numpy as np
import pytest
import torch

import gated_short_causal_amd as g
from oracle import hybrid as ho

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, I32 = torch.bfloat16, torch.int32
HALF = torch.finfo(BF).eps / 2


def _slack(q, k, D, scale):
    """Relative error of a probability from fp32 scores: the largest score's terms, times D + 8 roundings."""
    most = float(q.abs().max()) * float(k.abs().max()) * D * scale
    return (D + 8) * 2.0 ** -24 * (1 + most)


def _within(got, want, tol, what):
    got = got.detach().cpu().double().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} out of tolerance, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]} +- {np.broadcast_to(tol, bad.shape)[bad][0]}")


def _prompt_case(lens, Hq, Hkv, D, seed=0, lead=0, tail=0, amp=1.0):
    """Packed rows with `lead` and `tail` rows of no sequence; k and v are columns of one buffer."""
    gen = torch.Generator().manual_seed(seed)
    T = lead + sum(lens) + tail
    q = (torch.randn(T, Hq * D + 8, generator=gen) * amp).to(BF)[:, :Hq * D]
    kv = torch.randn(T, 2 * Hkv * D, generator=gen).to(BF)
    cu = torch.tensor([lead] + lens).cumsum(0).to(I32)
    return q, kv[:, :Hkv * D], kv[:, Hkv * D:], cu


def _run_prompt(q, k, v, cu, D, scale=None):
    T, W = q.shape
    out = torch.full((T, W + 16), float("nan"), dtype=BF, device=DEV)
    lse = torch.full((W // D, T), float("nan"), device=DEV)
    # keep the strides of the views on the device
    dq, dkv = q._base.to(DEV)[:, :W], k._base.to(DEV)
    n = k.shape[1]
    args = (dq, dkv[:, :n], dkv[:, n:], cu.to(DEV))
    g.lfm2sc_attn_prefill(*args, D, out[:, :W], lse=lse, scale=scale)
    return args, out, lse


def _untouched(x, rows):
    assert torch.isnan(x[rows].float()).all()


PROMPTS = [
    ([1], 1, 1, 64), ([1], 8, 2, 128), ([2, 1, 3], 4, 1, 64), ([63], 2, 2, 64), ([64], 2, 1, 128), ([65], 2, 1, 64),
    ([127, 1, 0, 128, 0], 4, 2, 64), ([129, 31, 97], 6, 2, 128), ([256], 4, 4, 64), ([257, 255], 3, 1, 64),
    ([500], 5, 5, 128), ([300, 2], 12, 1, 64), ([65] * 128, 16, 8, 64), ([33] * 260, 16, 8, 128), ([3] * 70 + [150] + [1] * 65, 2, 1, 64), ([700], 9, 3, 128), ([1111], 2, 1, 64),
]


@pytest.mark.parametrize("lens,Hq,Hkv,D", PROMPTS)
def test_prompt(lens, Hq, Hkv, D):
    q, k, v, cu = _prompt_case(lens, Hq, Hkv, D, seed=len(lens), lead=3, tail=5)
    scale = 0.2
    _, out, lse = _run_prompt(q, k, v, cu, D, scale)
    want, wlse, spread = ho.attention(q, k, v, cu, D, scale)
    rows = slice(int(cu[0]), int(cu[-1]))
    slack = _slack(q, k, D, scale)
    W = Hq * D
    _within(out[rows, :W], want[rows], HALF * (spread + np.abs(want))[rows] + slack * spread[rows], "out")
    _within(lse[:, rows], wlse[:, rows], slack * (1 + np.abs(wlse[:, rows])), "lse")
    for x in (out[:3], out[rows.stop:], out[:, W:], lse[:, :3], lse[:, rows.stop:]):
        assert torch.isnan(x.float()).all()


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_large_scores(D):
    """Scores of hundreds: the running maximum carries the softmax, most probabilities vanish."""
    q, k, v, cu = _prompt_case([400, 90], 4, 2, D, seed=9, amp=30.0)
    _, out, lse = _run_prompt(q, k, v, cu, D)
    want, wlse, spread = ho.attention(q, k, v, cu, D, D ** -0.5)
    slack = _slack(q, k, D, D ** -0.5)
    _within(out[:, :4 * D], want, HALF * (spread + np.abs(want)) + slack * spread, "out")
    _within(lse, wlse, slack * (1 + np.abs(wlse)), "lse")


def test_prompt_without_lse_and_repeats_bitwise():
    q, k, v, cu = _prompt_case([333, 64], 8, 2, 64, seed=2)
    args, out, _ = _run_prompt(q, k, v, cu, 64)
    again = torch.full_like(out, float("nan"))
    g.lfm2sc_attn_prefill(*args, 64, again[:, :512])
    assert torch.equal(out[:, :512].view(torch.int16), again[:, :512].view(torch.int16))


def test_prompt_keeps_a_nan_in_its_sequence():
    q, k, v, cu = _prompt_case([200, 100, 150], 2, 1, 64, seed=3)
    v._base[250] = float("nan")                      # k and v of row 50 of the second sequence
    _, out, _ = _run_prompt(q, k, v, cu, 64)
    assert torch.isfinite(out[:200, :128]).all() and torch.isfinite(out[300:, :128]).all()
    assert torch.isnan(out[250:300, :128]).all()


def test_prompt_offsets_past_32_bits():
    """70000 rows of 2^15 elements: the last rows lie past 2^31 elements."""
    T, stride, D = 70000, 1 << 15, 64
    gen = torch.Generator().manual_seed(4)
    big = torch.empty(T, stride, dtype=BF, device=DEV)
    small = torch.randn(150, 3 * 128, generator=gen).to(BF)
    big[-150:, :384] = small.to(DEV)
    out = torch.empty(T, stride, dtype=BF, device=DEV)
    cu = torch.tensor([T - 150, T], dtype=I32, device=DEV)
    lse = torch.empty(2, T, device=DEV)
    views = [big[:, i * 128:(i + 1) * 128] for i in range(3)]
    g.lfm2sc_attn_prefill(*views, cu, D, out[:, :128], lse=lse)
    ref = [small[:, i * 128:(i + 1) * 128] for i in range(3)]
    want, _, spread = ho.attention(*ref, [0, 150], D, 0.125)
    slack = _slack(ref[0], ref[1], D, 0.125)
    _within(out[-150:, :128], want, HALF * (spread + np.abs(want)) + slack * spread, "out")
    # and the backward, its gradients over the same offsets
    do = torch.randn(150, 128, generator=gen).to(BF)
    big[-150:, 512:640] = do.to(DEV)
    ws = torch.empty(g.lfm2sc_attn_backward_workspace_bytes(BF, D, 2, 2, T, 1), dtype=torch.uint8, device=DEV)
    grads = [out[:, 1024 * i:1024 * i + 128] for i in (1, 2, 3)]
    g.lfm2sc_attn_backward(*views, cu, D, out[:, :128], lse, big[:, 512:640], *grads, ws)
    want, bounds = ho.attention_backward(*ref, [0, 150], D, 0.125, do, HALF)
    for x, w, b, name in zip(grads, want, bounds, ("dq", "dk", "dv")):
        _within(x[-150:], w, b * (1 + 2 ** -6) + HALF * np.abs(w) + slack * b / HALF, name)


@pytest.mark.parametrize("lens,Hq,Hkv,D", PROMPTS)
def test_backward(lens, Hq, Hkv, D):
    q, k, v, cu = _prompt_case(lens, Hq, Hkv, D, seed=10 + len(lens), lead=2, tail=4)
    scale = 0.15
    args, out, lse = _run_prompt(q, k, v, cu, D, scale)
    T, W, n = q.shape[0], Hq * D, Hkv * D
    do = torch.randn(T, W, generator=torch.Generator().manual_seed(1)).to(BF)
    dq = torch.full((T, W), float("nan"), dtype=BF, device=DEV)
    dkv = torch.full((T, 2 * n + 8), float("nan"), dtype=BF, device=DEV)
    dk, dv = dkv[:, :n], dkv[:, n:2 * n]
    ws = torch.full((g.lfm2sc_attn_backward_workspace_bytes(BF, D, Hq, Hkv, T, len(lens)),), 255, dtype=torch.uint8, device=DEV)
    g.lfm2sc_attn_backward(*args, D, out[:, :W], lse, do.to(DEV), dq, dk, dv, ws, scale=scale)
    want, bounds = ho.attention_backward(q, k, v, cu, D, scale, do, HALF)
    rows = slice(int(cu[0]), int(cu[-1]))
    slack = _slack(q, k, D, scale)
    for x, w, b, name in zip((dq, dk, dv), want, bounds, ("dq", "dk", "dv")):
        # a second rounding on top of a first moves it by 1 + HALF; slack scales the same magnitudes as HALF does
        tol = b * (1 + 2 ** -6) + HALF * np.abs(w) + slack * b / HALF
        _within(x[rows], w[rows], tol[rows], name)
    for x in (dq[:2], dq[rows.stop:], dkv[:2], dkv[rows.stop:], dkv[:, 2 * n:]):
        assert torch.isnan(x.float()).all()
    again = [torch.empty(T, m, dtype=BF, device=DEV) for m in (W, n, n)]
    g.lfm2sc_attn_backward(*args, D, out[:, :W], lse, do.to(DEV), *again, ws, scale=scale)
    for x, y in zip((dq, dk, dv), again):
        assert torch.equal(x[rows].contiguous().view(torch.int16), y[rows].contiguous().view(torch.int16))


def test_backward_against_differences():
    """Directional derivatives of the forward's own output in fp64 differences (oracle forward, GPU gradient)."""
    D, Hq, Hkv = 64, 2, 1
    q, k, v, cu = _prompt_case([90, 40], Hq, Hkv, D, seed=21)
    do = torch.randn(130, Hq * D, generator=torch.Generator().manual_seed(2)).to(BF)
    args, out, lse = _run_prompt(q, k, v, cu, D)
    grads = [torch.empty(130, m, dtype=BF, device=DEV) for m in (Hq * D, D, D)]
    ws = torch.empty(g.lfm2sc_attn_backward_workspace_bytes(BF, D, Hq, Hkv, 130, 2), dtype=torch.uint8, device=DEV)
    g.lfm2sc_attn_backward(*args, D, out[:, :Hq * D], lse, do.to(DEV), *grads, ws)
    x = [t.double().numpy() for t in (q, k, v)]
    _, bounds = ho.attention_backward(q, k, v, cu, D, 0.125, do, HALF)
    rng = np.random.default_rng(3)
    for i in range(3):
        d = rng.normal(size=x[i].shape)
        eps = 1e-4
        f = [(ho.attention(*[x[j] + (s * eps * d if j == i else 0) for j in range(3)], cu, D, 0.125)[0] * do.double().numpy()).sum()
             for s in (1, -1)]
        got = grads[i].double().cpu().numpy()
        # the elements' roundings against the direction, all of one sign at worst
        tol = ((bounds[i] * (1 + 2 ** -6) + HALF * np.abs(got)) * np.abs(d)).sum()
        assert abs((got * d).sum() - (f[0] - f[1]) / (2 * eps)) < tol


def _pages(rng, N, lens, prefix, S, Hkv, D, spare=3, stride_heads=None):
    """Pools whose rows past the lengths, and spare pages, hold NaN."""
    most = max(1, -(-max(lens) // S))
    npp = -(-prefix // S)
    P = npp + N * most + spare
    pools = []
    order = torch.from_numpy(rng.permutation(P)).to(I32)
    pp, table = order[:npp], order[npp:npp + N * most].reshape(N, most)
    gen = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    kv = torch.full((P, S, 2, Hkv, D), float("nan"), dtype=BF)
    for j in range(npp):
        m = min(S, prefix - j * S)
        kv[pp[j], :m] = torch.randn(m, 2, Hkv, D, generator=gen).to(BF)
    for i in range(N):
        for j in range(most):
            m = min(S, lens[i] - j * S)
            if m > 0:
                kv[table[i, j], :m] = torch.randn(m, 2, Hkv, D, generator=gen).to(BF)
    return kv, pp.contiguous(), table.contiguous()


def _run_cached(q, kv, pp, prefix, table, lens, L, D, scale, split):
    Hq = q.shape[1] // D
    N, most = table.shape
    Hkv = kv.shape[3]
    dev = kv.to(DEV)
    k, v = (dev[:, :, 0], dev[:, :, 1]) if split else (dev[:, :, 0].contiguous(), dev[:, :, 1].contiguous())
    out = torch.full((N * L, Hq * D + 8), float("nan"), dtype=BF, device=DEV)
    ws = torch.full((g.lfm2sc_attn_cached_workspace_bytes(BF, D, Hq, Hkv, N, L, prefix, most, kv.shape[1]),), 255, dtype=torch.uint8,
                    device=DEV)
    g.lfm2sc_attn_cached(q.to(DEV), k, v, pp.to(DEV) if prefix else None, prefix, table.to(DEV), torch.tensor(lens, dtype=I32, device=DEV), L,
                         out[:, :Hq * D], ws, scale=scale)
    assert torch.isnan(out[:, Hq * D:].float()).all()
    return out[:, :Hq * D]


CACHED = [
    # lens, L, prefix, page, Hq, Hkv, D
    ([1], 1, 0, 16, 1, 1, 64), ([1], 1, 1, 16, 8, 2, 64), ([37], 1, 500, 16, 8, 2, 64), ([5, 64, 65, 200], 1, 63, 16, 8, 2, 64),
    ([33, 1, 129], 1, 64, 1, 4, 1, 128), ([8, 9, 300], 8, 65, 64, 10, 2, 128), ([20, 8], 8, 200, 8, 12, 1, 64),
    ([130] * 40, 1, 129, 32, 4, 4, 64), ([7, 31, 3], 3, 1000, 128, 5, 5, 128), ([0, 2, 5], 3, 0, 4, 4, 2, 64),
    ([0, 1, 0], 1, 0, 16, 4, 2, 128), ([0, 0], 2, 40, 16, 4, 2, 64), ([700, 1], 2, 300, 16, 2, 1, 64), ([2000], 1, 0, 64, 16, 2, 128),
    ([60] * 9, 5, 3000, 16, 8, 1, 64),
    # more workgroups than CUs, so never the direct form; without a prefix a single split writes the output itself
    ([0, 1, 300, 64, 65] * 30, 1, 700, 16, 4, 2, 64), ([0, 3, 130] * 30, 3, 0, 32, 8, 4, 128), ([1, 257] * 40, 1, 33, 8, 8, 8, 128),
    # the prefix's chunks end inside a tile
    ([2, 40], 2, 4500, 32, 8, 2, 64), ([9], 1, 6007, 1, 2, 1, 128),
]


@pytest.mark.parametrize("lens,L,prefix,S,Hq,Hkv,D", CACHED)
@pytest.mark.parametrize("split", [False, True])
def test_cached(lens, L, prefix, S, Hq, Hkv, D, split):
    rng = np.random.default_rng(len(lens) + L + prefix)
    N = len(lens)
    kv, pp, table = _pages(rng, N, lens, prefix, S, Hkv, D)
    q = torch.randn(N * L, Hq * D, generator=torch.Generator().manual_seed(5)).to(BF)
    scale = 0.2
    out = _run_cached(q, kv, pp, prefix, table, lens, L, D, scale, split)
    want, spread = ho.cached(q, kv[:, :, 0], kv[:, :, 1], pp, prefix, table, lens, L, scale)
    slack = _slack(q, torch.nan_to_num(kv.float()), D, scale)
    _within(out, want, HALF * (spread + np.abs(want)) + slack * spread, "out")


def test_cached_bad_numbers_stay_in_the_pool():
    """Page numbers outside the pool read the nearest page, lengths are clamped: the results are those of the clamped call."""
    rng = np.random.default_rng(1)
    kv, pp, table = _pages(rng, 2, [40, 40], 20, 16, 2, 64, spare=0)
    kv = torch.randn(kv.shape).to(BF)
    P = kv.shape[0]
    q = torch.randn(2, 128).to(BF)
    bad, fine = table.clone(), table.clone()
    bad[0, 1], fine[0, 1] = P + 1000, P - 1
    bad[1, 0], fine[1, 0] = -5, 0
    bp, fp = pp.clone(), pp.clone()
    bp[1], fp[1] = 1 << 30, P - 1
    a = _run_cached(q, kv, bp, 20, bad, [1 << 20, -3], 1, 64, None, False)
    b = _run_cached(q, kv, fp, 20, fine, [48, 0], 1, 64, None, False)
    assert torch.equal(a, b) and torch.isfinite(a).all()


def test_cached_pool_past_32_bits():
    """A pool of more than 2^32 elements a side, its last pages in use."""
    S, Hkv, D, stride, P = 64, 2, 64, 1 << 12, 17000
    pool = torch.empty(P, S, stride // 64, 64, dtype=BF, device=DEV)[:, :, :2]
    assert (P - 1) * S * stride > 1 << 32
    used = [P - 1, P - 2, 3, P - 5]
    small = torch.randn(4, S, 2, 64, generator=torch.Generator().manual_seed(1)).to(BF)
    for i, p in enumerate(used):
        pool[p] = small[i].to(DEV)
    q = torch.randn(1, 256, generator=torch.Generator().manual_seed(2)).to(BF)
    out = torch.empty(1, 256, dtype=BF, device=DEV)
    ws = torch.empty(g.lfm2sc_attn_cached_workspace_bytes(BF, D, 4, 2, 1, 1, 100, 2, S), dtype=torch.uint8, device=DEV)
    g.lfm2sc_attn_cached(q.to(DEV), pool, pool, torch.tensor(used[:2], dtype=I32, device=DEV), 100,
                         torch.tensor([used[2:]], dtype=I32, device=DEV), torch.tensor([99], dtype=I32, device=DEV), 1, out, ws)
    want, spread = ho.cached(q, small, small, [0, 1], 100, [[2, 3]], [99], 1, 0.125)
    slack = _slack(q, small, D, 0.125)
    _within(out, want, HALF * (spread + np.abs(want)) + slack * spread, "out")


def _draft_case(N, L, V, dtype, with_draft, seed, sharp=3.0, pad=0):
    rng = np.random.default_rng(seed)
    logits = rng.normal(size=(N, L + 1, V)) * sharp
    p = np.exp(logits - logits.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    noisy = logits[:, :L] + 0.7 * rng.normal(size=(N, L, V))
    q = np.exp(noisy - noisy.max(-1, keepdims=True))
    q /= q.sum(-1, keepdims=True)
    tokens = np.array([[rng.choice(V, p=q[n, s]) if with_draft else q[n, s].argmax() for s in range(L)] for n in range(N)])
    tokens = torch.from_numpy(tokens.reshape(N, L)).to(I32)

    def rows(x):
        full = torch.full((x.shape[0] * x.shape[1], V + pad), float("nan"), dtype=dtype)
        full[:, :V] = torch.from_numpy(x.reshape(-1, V)).to(dtype)
        return full[:, :V]

    ua = torch.from_numpy(rng.random((N, L))).float().clamp(max=1 - 2 ** -24)
    us = torch.from_numpy(rng.random(N)).float().clamp(max=1 - 2 ** -24)
    return rows(p), rows(q) if with_draft and L else None, tokens, ua, us


def _dev(x):
    return None if x is None else (x if x._base is None else x._base).to(DEV)[:, :x.shape[1]]


def _run_drafts(target, draft, tokens, ua, us, num_drafts=None):
    N, L = tokens.shape
    V = target.shape[1]
    a, keep, nxt = (torch.full((N,), -77, dtype=I32, device=DEV) for _ in range(3))
    ws = torch.full((g.lfm2sc_accept_drafts_workspace_bytes(N, L, V),), 255, dtype=torch.uint8, device=DEV)
    g.lfm2sc_accept_drafts(_dev(target), tokens.to(DEV), ua.to(DEV), us.to(DEV), a, nxt, ws, draft_probs=_dev(draft),
                           num_drafts=None if num_drafts is None else num_drafts.to(DEV), keep_len=keep)
    assert torch.equal(keep, a + 1)
    return a.cpu().numpy(), nxt.cpu().numpy()


def _check_drafts(*args, num_drafts=None):
    a, nxt = _run_drafts(*args, num_drafts=num_drafts)
    target, draft, tokens, ua, us = args
    wa, wn = ho.accept_drafts(target, tokens, ua, us, draft, None if num_drafts is None else num_drafts.numpy())
    assert (a == wa).all(), (a, wa)
    assert (nxt == wn).all(), (nxt, wn)
    return a


@pytest.mark.parametrize("N,L,V,pad", [(1, 1, 1, 0), (3, 2, 7, 1), (5, 7, 8, 0), (2, 0, 100, 3), (4, 64, 33, 0), (9, 4, 2048, 0),
                                       (3, 4, 4097, 0), (70, 3, 1000, 5), (2, 8, 32003, 0), (1, 5, 65536, 8),
                                       (40, 2, 8193, 0), (3, 3, 70001, 0), (2, 1, 131072, 1), (34, 1, 66001, 0), (1, 1, 600000, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("with_draft", [True, False])
def test_drafts(N, L, V, pad, dtype, with_draft):
    _check_drafts(*_draft_case(N, L, V, dtype, with_draft, seed=N + L + V, pad=pad))


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("V", [5000, 70000])
def test_drafts_borders(dtype, V):
    """u of 0, of just below 1 and outside [0, 1); a NaN u; drafts outside the vocabulary; ragged numbers of drafts."""
    target, draft, tokens, ua, us = _draft_case(12, 3, V, dtype, True, seed=8)
    us[:6] = torch.tensor([0.0, 1 - 2 ** -24, 1.0, 2.0, -1.0, float("nan")])
    ua[6] = 0.0
    ua[7] = 1.0
    ua[8, 1] = float("nan")
    tokens[9, 0], tokens[10, 1], tokens[11, 2] = -1, V, 1 << 30
    ua[10, 0], ua[11, :2] = 0.0, 0.0
    _check_drafts(target, draft, tokens, ua, us)
    _check_drafts(target, None, tokens, ua, us)
    nd = torch.tensor([0, 1, 2, 3, 4, -1, 3, 2, 1, 1, 2, 100], dtype=I32)
    _check_drafts(target, draft, tokens, ua, us, num_drafts=nd)


@pytest.mark.parametrize("V", [16, 9001, 80003])
def test_drafts_degenerate_rows(V):
    """p = q (nothing left: drawn from p), one-hot rows, all-zero rows, NaN and negative entries, flat rows with the
    border on a token's edge."""
    N, L = 8, 1
    target, draft = torch.zeros(2 * N, V), torch.zeros(N, V)
    r = torch.rand(V, generator=torch.Generator().manual_seed(1))
    target[0], draft[0] = r, r                       # rejected by u = 1: the residual is empty
    target[2, 3], draft[1, 5] = 1.0, 1.0             # one-hot, elsewhere
    target[4], draft[2] = 0.0, r                     # nothing in the target
    target[6], draft[3] = r, r.flip(0)
    target[6, ::3] = float("nan")
    target[8], draft[4] = -r, r
    target[8, 7] = 0.25
    target[10], draft[5] = 1.0 / 16, 0.0             # flat: u sum falls on edges
    target[12, V - 1], draft[6] = 1e-38, 0.0         # only the last token, tiny
    target[14], target[15], draft[7] = r, r, 0.0
    tokens = torch.tensor([[1], [5], [2], [0], [3], [4], [0], [2]], dtype=I32)
    ua = torch.ones(N, 1)
    ua[7] = 0.0                                      # accepted: the bonus row
    for u in (0.0, 0.25, 0.5, 0.9375, 1 - 2 ** -24):
        us = torch.full((N,), u)
        _check_drafts(target, draft, tokens, ua, us)
        _check_drafts(target, None, tokens, ua, us)


def test_speculative_step_end_to_end():
    """verify_window -> accept_drafts -> commit_window: keep_len picks the tape's window on the device."""
    N, L, H, K, V, slots = 6, 4, 64, 3, 500, 9
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(N * (L + 1), 3 * H, generator=gen).to(BF).to(DEV)
    w = (torch.rand(H, K, generator=gen) - 0.5).to(BF).to(DEV)
    pool = torch.randn(slots, H, K, generator=gen).to(BF).to(DEV)
    slot = torch.tensor([8, 0, 3, 5, 1, 6], dtype=I32, device=DEV)
    win = torch.empty(N, L + 1, H, K, dtype=BF, device=DEV)
    y = torch.empty(N * (L + 1), H, dtype=BF, device=DEV)
    g.lfm2sc_verify_window(x, w, pool, slot, L + 1, win, y)
    target, draft, tokens, ua, us = _draft_case(N, L, V, torch.float32, True, seed=4, sharp=1.0)
    a, keep, nxt = (torch.empty(N, dtype=I32, device=DEV) for _ in range(3))
    ws = torch.empty(g.lfm2sc_accept_drafts_workspace_bytes(N, L, V), dtype=torch.uint8, device=DEV)
    g.lfm2sc_accept_drafts(target.to(DEV), tokens.to(DEV), ua.to(DEV), us.to(DEV), a, nxt, ws, draft_probs=draft.to(DEV), keep_len=keep)
    before = pool.clone()
    g.lfm2sc_commit_window(win, keep, pool, slot)
    wa, _ = ho.accept_drafts(target, tokens, ua, us, draft)
    assert len(set(wa.tolist())) > 1
    for i in range(N):
        assert torch.equal(pool[slot[i].item()], win[i, wa[i]])
    rest = [s for s in range(slots) if s not in slot.tolist()]
    assert torch.equal(pool[rest], before[rest])


def _replay(call, outs, inputs):
    """Three replays of a captured call on changed inputs, each against the eager call's bits."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for x in inputs:
            x.copy_(torch.randn(x.shape, device=DEV).abs().to(x.dtype))
        call()
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, want):
            assert torch.equal(o, e)


def test_graph_replays():
    D, Hq, Hkv, T = 64, 4, 2, 200
    q, k, v, do = (torch.randn(T, n * D, device=DEV).to(BF) for n in (Hq, Hkv, Hkv, Hq))
    cu = torch.tensor([0, 77, T], dtype=I32, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(Hq, T, device=DEV)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(g.lfm2sc_attn_backward_workspace_bytes(BF, D, Hq, Hkv, T, 2), dtype=torch.uint8, device=DEV)

    def train():
        g.lfm2sc_attn_prefill(q, k, v, cu, D, out, lse=lse)
        g.lfm2sc_attn_backward(q, k, v, cu, D, out, lse, do, dq, dk, dv, ws)

    _replay(train, (out, lse, dq, dk, dv), (q, k, v, do))

    pool = torch.randn(30, 16, Hkv, D, device=DEV).to(BF)
    pp, table = torch.arange(4, dtype=I32, device=DEV), torch.arange(4, 16, dtype=I32, device=DEV).reshape(3, 4)
    lens = torch.tensor([3, 40, 64], dtype=I32, device=DEV)
    cq, cout = torch.randn(6, Hq * D, device=DEV).to(BF), torch.empty(6, Hq * D, dtype=BF, device=DEV)
    cws = torch.empty(g.lfm2sc_attn_cached_workspace_bytes(BF, D, Hq, Hkv, 3, 2, 60, 4, 16), dtype=torch.uint8, device=DEV)
    _replay(lambda: g.lfm2sc_attn_cached(cq, pool, pool, pp, 60, table, lens, 2, cout, cws), (cout,), (cq, pool))

    target, draft = torch.rand(9, 5001, device=DEV), torch.rand(6, 5001, device=DEV)
    tokens = torch.randint(0, 5001, (3, 2), device=DEV).to(I32)
    ua, us = torch.rand(3, 2, device=DEV), torch.rand(3, device=DEV)
    a, nxt = torch.empty(3, dtype=I32, device=DEV), torch.empty(3, dtype=I32, device=DEV)
    dws = torch.empty(g.lfm2sc_accept_drafts_workspace_bytes(3, 2, 5001), dtype=torch.uint8, device=DEV)
    _replay(lambda: g.lfm2sc_accept_drafts(target, tokens, ua, us, a, nxt, dws, draft_probs=draft), (a, nxt), (target, draft))


def test_another_stream():
    """Work queued on a side stream runs there, after what was queued on it."""
    q, k, v, cu = _prompt_case([500], 8, 2, 64, seed=7)
    args, out, _ = _run_prompt(q, k, v, cu, 64)
    side = torch.cuda.Stream()
    late = [torch.zeros_like(x) for x in args[:3]]
    got = torch.empty_like(out)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for x, y in zip(late, args):
            x.copy_(y)
        g.lfm2sc_attn_prefill(*late, args[3], 64, got[:, :512])
    side.synchronize()
    assert torch.equal(out[:, :512], got[:, :512])


def test_example_runs_them_together():
    from examples import hybrid_step
    dev = torch.device(DEV)
    torch.manual_seed(0)
    for x in hybrid_step.train_step([70, 1, 130], dev).values():
        assert torch.isfinite(x.float()).all()
    s = hybrid_step.speculative_step(5, 3, 100, dev, vocab=300)
    assert torch.isfinite(s["out"].float()).all()
    for i, a in enumerate(s["accepted"].tolist()):
        assert 0 <= a <= 3 and 0 <= s["next"][i] < 300
        assert torch.equal(s["pool"][s["slots"][i].item()], s["tape"][i, a])


_CHECK_SCRIPT = """
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

x = torch.randn(20, 128, device=d).to(BF)
out, lse = torch.empty_like(x), torch.empty(2, 20, device=d)
def prompt(*cu):
    return status(lambda: g.lfm2sc_attn_prefill(x, x, x, ints(*cu), 64, out, lse=lse))
pool = torch.randn(8, 16, 2, 64, device=d).to(BF)
def cached(pp, table, n):
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=d)
    return status(lambda: g.lfm2sc_attn_cached(x[:1], pool, pool, ints(pp), 10, ints(table).reshape(1, 1), ints(n), 1, out[:1], ws))
p, u, r = torch.rand(2, 50, device=d), torch.rand(1, 1, device=d), torch.empty(2, dtype=I32, device=d)
def drafts(token, n):
    ws = torch.empty(1 << 12, dtype=torch.uint8, device=d)
    return status(lambda: g.lfm2sc_accept_drafts(p, ints(token).reshape(1, 1), u, u[0], r[:1], r[1:], ws, num_drafts=ints(n)))
s = [prompt(0, 5, 20), prompt(0, 21), prompt(7, 3), cached(1, 2, 16), cached(8, 2, 16), cached(1, -1, 16), cached(1, 2, 17),
     drafts(49, 1), drafts(50, 1), drafts(0, 2)]
torch.cuda.synchronize()
print("STATUS", s)
"""


def test_check_mode_reports_bad_device_data():
    """LFM2SC_CHECK=1 (read once per process, hence a child) turns row offsets, pages, lengths, tokens and numbers of drafts
    out of range into LFM2SC_ERR_PRECONDITION (6)."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _CHECK_SCRIPT, root], env=dict(os.environ, LFM2SC_CHECK="1"), capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    line = [x for x in r.stdout.splitlines() if x.startswith("STATUS")][0]
    assert line == "STATUS [0, 6, 6, 0, 6, 6, 6, 0, 6, 6]", line
