"""Attention over the 8-bit cache where many query rows share a prefix (GPU): the form whose workgroups stage the prefix's tiles for
128 rows, at every tail of a prefix, with as many tiles to a workgroup as its pipeline needs to repeat itself, and joins of more
than 64 parts.  Each test asks the library's plan that its sizes take the form that it is about.  The reference is the formula
in fp64 on the GPU, pinned to the oracle; tolerance as in test_gpu_cache8."""
import numpy as np
import pytest
import torch

import gated_short_causal_amd as g
from oracle import cache8 as o8
from test_cache8_workspace import SHARED, SPLIT, plan
from test_gpu_cache8 import BF, DEV, Cache, _attend, _close
from test_gpu_cache8_more import _setup

pytestmark = pytest.mark.gpu
# every instance of the kernel's two formats and two kinds of scale, in pages below and above a tile
KINDS = [("e4m3", 16, 16), ("e4m3", 128, 1), ("int8", 128, 64), ("int8", 16, 1)]


def _values(c, pages, n):
    """k, v [n, heads, D] in float64 on the GPU of the first n tokens of a list of pages."""
    _, H, S, D, B = c.shape
    p = torch.as_tensor(np.asarray(pages[:-(-n // S)]), dtype=torch.long)
    out = []
    for codes, scales in (("k", "ks"), ("v", "vs")):
        x, s = torch.from_numpy(c.host[codes])[p].to(DEV), torch.from_numpy(c.host[scales])[p].to(DEV).double()
        x = x * s.repeat_interleave(B, 2)[..., None]
        out.append(x.transpose(1, 2).reshape(-1, H, D)[:n])
    return out


def _reference(c, q, pp, prefix, table, lens, L, scale):
    """As oracle.cache8.attention: out, sum p |v|, and the largest sum of a score's magnitudes."""
    _, H, S, D, _ = c.shape
    N, G = len(lens), q.shape[1] // (H * D)
    x = q.to(DEV).double().reshape(N, L, H, G, D)
    pk, pv = _values(c, pp, prefix)
    out, spread = (torch.zeros(N, L, H, G, D, dtype=torch.float64, device=DEV) for _ in range(2))
    most = 0.0
    first = []
    for h in range(H):
        rows = x[:, :, h].reshape(N * L * G, D)
        first.append((scale * rows @ pk[:, h].T).reshape(N, L * G, prefix))
        most = max(most, float((rows.abs() @ pk[:, h].abs().T).max()) * scale)
    suffixes = {}
    for i, n in enumerate(lens):
        pages = tuple(table[i])
        if pages not in suffixes:
            suffixes[pages] = _values(c, pages, len(pages) * S)
        k, v = (y[:n] for y in suffixes[pages])
        seen = torch.arange(n, device=DEV) <= n - L + torch.arange(L, device=DEV)[:, None]       # [L, n]
        for h in range(H):
            rows = x[i, :, h].reshape(L * G, D)
            own = (scale * rows @ k[:, h].T).masked_fill(~seen.repeat_interleave(G, 0), -float("inf"))
            p = torch.softmax(torch.cat([first[h][i], own], 1), 1)
            out[i, :, h] = (p[:, :prefix] @ pv[:, h] + p[:, prefix:] @ v[:, h]).reshape(L, G, D)
            spread[i, :, h] = (p[:, :prefix] @ pv[:, h].abs() + p[:, prefix:] @ v[:, h].abs()).reshape(L, G, D)
            if n:
                most = max(most, float((rows.abs() @ k[:, h].abs().T).max()) * scale)
    return out.reshape(N * L, -1).cpu().numpy(), spread.reshape(N * L, -1).cpu().numpy(), most


def _make(fmt, S, B, D, Hkv, N, L, prefix, own, seed, late=False):
    """A cache of a prefix and four suffixes that the sequences share, in pages out of order; page numbers and lengths.  late:
    keys grow along the prefix, so that the rows' maxima keep moving to later tiles."""
    npre, most = -(-prefix // S), -(-own // S)
    P = npre + 4 * most
    c = Cache(fmt, P, Hkv, S, D, B, seed=seed)
    order = np.random.default_rng(seed).permutation(P).astype(np.int32)
    pp, suffixes = order[:npre], order[npre:].reshape(4, most)
    if late:
        at = (torch.arange(npre, dtype=torch.float64)[:, None] * S + torch.arange(S // B) * B) / prefix
        grown = (0.2 + 3 * at ** 3 + 3 * (at > 0.98)).float().to(DEV)
        c.args[2][torch.from_numpy(pp).long().to(DEV)] *= grown[:, None]
        c.host = c.read()
    lens = [(7 * i) % (own - L + 1) + L for i in range(N)]
    lens[0], lens[1] = own, L - 1
    return c, pp, np.stack([suffixes[i % 4] for i in range(N)]), lens


def _spoil(c, pp, prefix):
    """NaN for the codes (e4m3) and scales behind the prefix's end."""
    _, _, S, _, B = c.shape
    k, v, ks, vs = c.args
    for t in range(prefix, len(pp) * S):
        page = int(pp[t // S])
        if c.fmt == "e4m3":
            k.view(torch.int8)[page, :, t % S] = 0x7f
            v.view(torch.int8)[page, :, t % S // 16, :, t % 16] = 0x7f
        if t % B == 0:
            ks[page, :, t % S // B] = float("nan")
            vs[page, :, t % S // B] = float("nan")


def _query(rows, width):
    return torch.randn(rows, width, generator=torch.Generator().manual_seed(1)).to(BF)


def _run(c, q, pp, prefix, table, lens, L, what="", **kw):
    want = _reference(c, q, pp, prefix, table, lens, L, kw.get("scale", c.shape[3] ** -0.5))
    _spoil(c, pp, prefix)
    got = _attend(c, q, pp, prefix, table, lens, L, **kw)
    _close(got, want, what)
    assert torch.equal(got, _attend(c, q, pp, prefix, table, lens, L, **kw))


def test_the_reference_is_the_oracle():
    c, pp, table, lens = _make("int8", 16, 16, 64, 2, 5, 3, 70, 40, 3)
    q = _query(15, 2 * 2 * 64)
    a, b = _reference(c, q, pp, 70, table, lens, 3, 0.125), o8.attention(q, c.host, pp, 70, table, lens, 3, 0.125)
    for x, y in zip(a, b):
        np.testing.assert_allclose(x, y, rtol=1e-11, atol=1e-13)


@pytest.mark.parametrize("fmt,S,B", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,L,G", [(128, 1, 2), (129, 1, 1), (70, 9, 2)])
@pytest.mark.parametrize("prefix", [1, 63, 64, 65, 200, 511])
def test_every_tail(prefix, N, L, G, D, fmt, S, B):
    """Prefixes of one to eight tiles that end anywhere in one; rows that fill their last workgroup, or one row of it."""
    Hkv, own = 8, 30
    assert plan(D, Hkv * G, Hkv, N, L, prefix, own).form == SHARED
    c, pp, table, lens = _make(fmt, S, B, D, Hkv, N, L, prefix, own, prefix + N)
    _run(c, _query(N * L, Hkv * G * D), pp, prefix, table, lens, L, max_suffix_len=own)


@pytest.mark.parametrize("fmt,S,B", KINDS)
@pytest.mark.parametrize("D,G,Hkv,N,L,prefix,own,tiles", [
    (64, 4, 8, 256, 1, 3839, 40, 5), (64, 4, 8, 256, 1, 4499, 40, 6), (64, 4, 8, 256, 1, 5121, 40, 7), (64, 5, 8, 64, 8, 5057, 90, 20),
    (64, 1, 32, 43, 3, 9000, 20, 12), (128, 1, 16, 129, 1, 4500, 40, 5), (128, 1, 16, 129, 1, 5121, 40, 6), (128, 5, 8, 16, 8, 5130, 40, 7),
    (128, 5, 8, 64, 8, 3823, 90, 20), (128, 2, 8, 70, 1, 9000, 30, 5)])
def test_many_tiles_to_a_workgroup(D, G, Hkv, N, L, prefix, own, tiles, fmt, S, B):
    """Chains of 5 tiles and more: page numbers are looked up four tiles ahead and buffers come round twice."""
    p = plan(D, Hkv * G, Hkv, N, L, prefix, own)
    assert p.form == SHARED and p.prefix_chunk == 64 * tiles
    c, pp, table, lens = _make(fmt, S, B, D, Hkv, N, L, prefix, own, tiles, late=True)
    _run(c, _query(N * L, Hkv * G * D), pp, prefix, table, lens, L, max_suffix_len=own)


@pytest.mark.parametrize("fmt,S,B", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,form", [(1, SPLIT), (20, SHARED)])
def test_more_than_64_parts(N, form, D, fmt, S, B):
    Hkv, G, prefix, own = 1, 8, 32700, 40
    p = plan(D, G, Hkv, N, 1, prefix, own)
    assert p.form == form and p.prefix_splits + p.suffix_splits > 128
    npre, most = -(-prefix // S), -(-own // S)
    c = Cache(fmt, npre + most, Hkv, S, D, B, seed=N)
    order = np.random.default_rng(N).permutation(npre + most).astype(np.int32)
    pp, table, lens = order[:npre], np.repeat(order[None, npre:], N, 0), [own - i for i in range(N)]
    _run(c, _query(N, G * D), pp, prefix, table, lens, 1, max_suffix_len=own)


@pytest.mark.parametrize("B", [1, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_a_tiny_scale(D, B):
    """Scores that underflow, of blocks of zeros among them, weigh alike, and keys past the end nothing."""
    Hkv, G, N, L, prefix, own, S = 2, 2, 70, 2, 2100, 21, 32
    assert plan(D, Hkv * G, Hkv, N, L, prefix, own).form == SHARED
    for scale in (1e-12, 1e-38):
        c, pp, table, lens = _make("int8", S, B, D, Hkv, N, L, prefix, own, N)
        c.args[2][::2] = 0.
        c.host = c.read()
        _run(c, _query(N * L, Hkv * G * D), pp, prefix, table, lens, L, max_suffix_len=own, scale=scale)


def test_a_nan_query_stays_in_its_row():
    c, rows, lens, pos, out, step = _setup(N=70, L=2, prefix=2200)
    assert plan(64, 8, 2, 70, 2, 2200, 64).form == SHARED
    step()
    torch.cuda.synchronize()
    before = out.clone()
    rows[5, :64] = float("nan")                              # one head of one row's query
    step()
    torch.cuda.synchronize()
    assert torch.isnan(out[5, :64].float()).all()
    out[5, :64] = before[5, :64]
    assert torch.equal(out, before)


def test_a_captured_step_replays():
    """Rotate, write and attend in one graph, with eager steps and synchronizations between the replays."""
    c, rows, lens, pos, out, step = _setup(N=80, prefix=2200, limit=500)
    assert plan(64, 8, 2, 80, 2, 2200, 512).form == SHARED
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(4):
        rows.normal_()
        lens.add_(2)
        pos.add_(2)
        codes, scales = c.codes.clone(), c.scales.clone()
        step()
        torch.cuda.synchronize()
        want, wc, wsc = out.clone(), c.codes.clone(), c.scales.clone()
        c.codes.copy_(codes)
        c.scales.copy_(scales)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(c.codes, wc) and torch.equal(c.scales, wsc), r
