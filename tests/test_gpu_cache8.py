"""The 8-bit cache on the GPU: codes and scales against the oracle bit for bit, values read back bit for bit, and attention
over it against fp64.

Tolerance of the attention: out = sum w v' / sum w / vs with w = p vs rounded to bf16 (v' the code, vs its scale), so a row's
probabilities p are p (1 + d), |d| <= HALF, above and below: sum p d (v - out) <= HALF (sum p |v| + |out|), and the output's own
rounding HALF |out| more.  1 / vs is held as two bf16 numbers, 2^-16 off; that and products of errors are the factor 1 + 2^-7.
fp32: D products summed and a few more roundings of a score move it by at most (D + 10) 2^-24 of its terms' magnitudes, hence a
probability relatively by as much (D is at most 128), again above and below: twice that of sum p |v|, as |out| is below it.
"""
import numpy as np
import pytest
import torch

import gated_short_causal_amd as g
from oracle import cache8 as o8

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
HALF = torch.finfo(BF).eps / 2
E4M3 = torch.float8_e4m3fn
FORMATS = {"int8": torch.int8, "e4m3": E4M3}


class Cache:
    """Pools on the GPU (k and v pages and scales in one buffer each, with room between pages) and the oracle's copy."""

    def __init__(self, fmt, P, H, S, D, B, seed=0, full=True):
        self.fmt, self.shape = fmt, (P, H, S, D, B)
        gen = torch.Generator().manual_seed(seed)
        page, n = H * S * D, H * (S // B)
        if fmt == "int8":
            codes = torch.randint(-127, 128, (P, 2 * page + 32), generator=gen).to(torch.int8)
        else:
            codes = (torch.randn(P, 2 * page + 32, generator=gen) * 60).clamp(-448, 448).to(E4M3).view(torch.int8)
        scales = torch.rand(P, 2 * n + 3, generator=gen) * 0.02 + 0.001
        if not full:                                         # nothing written yet: NaN codes (e4m3) and scales
            codes.fill_(0x7f)
            scales.fill_(float("nan"))
        self.codes, self.scales = codes.to(DEV), scales.to(DEV)
        dt = FORMATS[fmt]
        self.args = (self.codes[:, :page].view(dt).unflatten(1, (H, S, D)),
                     self.codes[:, page:2 * page].view(dt).unflatten(1, (H, S // 16, D, 16)),
                     self.scales[:, :n].unflatten(1, (H, S // B)), self.scales[:, n:2 * n].unflatten(1, (H, S // B)))
        self.host = self.read()

    def read(self):
        P, H, S, D, B = self.shape
        page, n = H * S * D, H * (S // B)
        v = self.codes.cpu()[:, :2 * page].contiguous().view(FORMATS[self.fmt]).double()
        s = self.scales.cpu()
        return {"page": S, "block": B, "int8": self.fmt == "int8", "k": v[:, :page].reshape(P, H, S, D).numpy().copy(),
                "v": v[:, page:].reshape(P, H, S // 16, D, 16).transpose(3, 4).reshape(P, H, S, D).numpy().copy(),
                "ks": s[:, :n].reshape(P, H, S // B).numpy().copy(), "vs": s[:, n:2 * n].reshape(P, H, S // B).numpy().copy()}

    def check(self, what=""):
        got = self.read()
        for name in ("ks", "vs", "k", "v"):
            same = (got[name] == self.host[name]) | (np.isnan(got[name]) & np.isnan(self.host[name]))
            assert same.all(), (f"{what} {name}: {(~same).sum()} of {same.size} differ, first at {np.argwhere(~same)[0]}: "
                                f"{got[name][~same][0]!r} for {self.host[name][~same][0]!r}")


def _kv(T, H, D, dtype, seed, amp=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, 2 * H * D + 8, generator=gen) * torch.exp(torch.randn(T, 1, generator=gen)) * amp
    return x.to(dtype)


def _write(c, x, table, seq_len, lens, uniform=False, lead=0, tail=0):
    P, H, S, D, B = c.shape
    y = torch.cat([x.new_full((lead, x.shape[1]), float("nan")), x, x.new_full((tail, x.shape[1]), float("nan"))]).to(DEV)
    cu = None if uniform else torch.tensor([lead] + lens).cumsum(0).to(I32).to(DEV)
    g.lfm2sc_cache8_write(y[:, :H * D], y[:, H * D:2 * H * D], *c.args, torch.from_numpy(table).to(DEV), torch.tensor(seq_len, dtype=I32, device=DEV),
                          cu_seqlens=cu)
    torch.cuda.synchronize()
    o8.write(c.host, x[:, :H * D], x[:, H * D:2 * H * D], table, seq_len, lens)


def _table(N, most, P, seed=0):
    return np.random.default_rng(seed).permutation(P)[:N * most].reshape(N, most).astype(np.int32)


GEOMETRY = [(16, 1), (16, 16), (32, 16), (64, 32), (64, 64), (128, 128), (256, 64), (128, 1)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S,B", GEOMETRY)
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_write_packed(fmt, S, B, D, dtype):
    """Sequences that begin, continue within a block, end inside tiles, hold nothing, or have rows before token 0."""
    H, N, most = 3, 7, 3
    most = max(most, -(-300 // S))
    c = Cache(fmt, N * most + 2, H, S, D, B, seed=S + B)
    table = _table(N, most, N * most + 2)
    lens = [1, 0, 2 * S + 3 if 2 * S + 3 < 200 else 150, 17, 5, 40, 33]
    held = [0, 9, 0, 15, B, S - 1 if S < 200 else 77, -7]
    _write(c, _kv(sum(lens), H, D, dtype, 1), table, [a + b for a, b in zip(held, lens)], lens, lead=2, tail=3)
    c.check(f"{fmt} {S} {B}")


@pytest.mark.parametrize("L", [1, 2, 8, 19])
@pytest.mark.parametrize("S,B,D", [(16, 16, 64), (16, 1, 128), (64, 64, 128), (128, 128, 64), (32, 1, 64)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_write_step_by_step(fmt, S, B, D, L):
    """Steps of L tokens, of growing and of falling size: scales grow by powers of two and earlier codes follow."""
    H, N, most = 2, 3, max(2, 128 // S)
    c = Cache(fmt, N * most, H, S, D, B, full=False)
    table = _table(N, most, N * most)
    at = [0, 5, 14]
    # the first tokens of sequences 1 and 2
    first = _kv(19, H, D, BF, 2)
    _write(c, first, table, at, [0, 5, 14])
    kept = {}
    for step in range(5):
        amp = [1.0, 0.01, 30.0, 3.0, 1000.0][step]
        at = [a + L for a in at]
        if max(at) > most * S:
            break
        _write(c, _kv(N * L, H, D, BF, 10 + step, amp), table, at, [L] * N, uniform=True)
        c.check(f"step {step}")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_values_stay_within_one_step(fmt):
    """However many tokens join a block: a kept value is at most one step (e4m3: of its own size) from what was written."""
    H, S, D, B = 1, 64, 64, 64
    c = Cache(fmt, 1, H, S, D, B, full=False)
    table = np.zeros((1, 1), dtype=np.int32)
    rows = []
    for t in range(64):
        x = _kv(1, H, D, F32, 100 + t, 1.3 ** t * 1e-3)
        rows.append(x[:, :D].double().numpy())
        _write(c, x, table, [t + 1], [1], uniform=True)
    c.check()
    x, scale = np.concatenate(rows), float(c.host["ks"][0, 0, 0])
    got = c.host["k"][0, 0] * scale
    if fmt == "int8":
        assert (np.abs(got - x) <= scale * (1 + 2.0 ** -20)).all()
    else:
        # powers of two: only values below the smallest normal code lose digits again
        assert (np.abs(got - x) <= np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -9)).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_write_odd_values(fmt):
    """Zeros, tiny and huge values, infinities and NaN, and blocks that begin with them."""
    H, S, D, B, N = 1, 32, 64, 16, 8
    c = Cache(fmt, N, H, S, D, B, full=False)
    table = np.arange(N, dtype=np.int32)[:, None]
    x = _kv(N * 5, H, D, F32, 3).reshape(N, 5, -1)
    x[0] = 0.0
    x[1] *= 1e-37
    x[2] *= 1e36
    x[3, 1, 3], x[3, 2, 70] = float("inf"), -float("inf")
    x[4, :, :] = float("nan")
    x[5, 2, 9], x[5, 2, 80] = float("nan"), float("nan")
    x[6, :, ::2] = 0.0
    x[7] = float("inf")
    _write(c, x.reshape(N * 5, -1), table, [5] * N, [5] * N, uniform=True)
    c.check("first")
    y = _kv(N * 3, H, D, F32, 4).reshape(N, 3, -1)
    y[2] *= 1e-30
    y[6] = 0.0
    _write(c, y.reshape(N * 3, -1), table, [8] * N, [3] * N, uniform=True)
    c.check("joined")


def test_write_leaves_bad_pages_and_other_tokens_alone():
    H, S, D, B, N, P = 2, 16, 64, 16, 4, 5
    c = Cache("int8", P, H, S, D, B, seed=3)
    table = np.array([[4, 99], [-1, 2], [0, 1 << 30], [-(1 << 31), 3]], dtype=np.int32)
    before, scales = c.codes.clone(), c.scales.clone()
    _write(c, _kv(N * 20, H, D, BF, 8), table, [20, 20, 20, 20], [20] * N, uniform=True)
    c.check()
    page = H * S * D
    assert torch.equal(c.codes[:, 2 * page:], before[:, 2 * page:]) and torch.equal(c.codes[1], before[1])
    assert torch.equal(c.scales[1], scales[1]) and torch.equal(c.scales[:, 4:], scales[:, 4:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S,B", GEOMETRY)
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_read(fmt, S, B, D, dtype):
    H, N, most, lead, tail = 3, 6, max(2, -(-130 // S)), 2, 3
    c = Cache(fmt, N * most, H, S, D, B, seed=5)
    table = _table(N, most, N * most, 1)
    table[1, 0], table[2, 0] = -3, 1 << 30
    lens, seq_len = [130, 1, 17, 0, 16, 9], [130, S + 1, 30, 50, 32, 4]
    T = lead + sum(lens) + tail
    cu = torch.tensor([lead] + lens).cumsum(0).to(I32)
    out = torch.full((T, 2 * H * D + 8), float("nan"), dtype=dtype, device=DEV)
    g.lfm2sc_cache8_read(*c.args, torch.from_numpy(table).to(DEV), torch.tensor(seq_len, dtype=I32, device=DEV), out[:, :H * D],
                         out[:, H * D:2 * H * D], cu_seqlens=cu.to(DEV))
    want = torch.full((T, 2 * H * D + 8), float("nan"), dtype=F32)
    for i, n in enumerate(lens):
        k, v = o8.values(c.host, table[i], seq_len[i])
        rows = np.concatenate([k.reshape(seq_len[i], -1), v.reshape(seq_len[i], -1)], 1)
        m = min(n, seq_len[i])                               # rows before token 0 are left alone
        want[cu[i] + n - m:cu[i] + n, :2 * H * D] = torch.from_numpy(rows[seq_len[i] - m:]).float()
    want = want.to(dtype)
    got = out.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(), want.nan_to_num())


def test_write_then_read_uniform():
    H, S, D, B, N, L = 8, 64, 128, 32, 5, 37
    c = Cache("e4m3", 2 * N, H, S, D, B, full=False)
    table = torch.from_numpy(_table(N, 2, 2 * N)).to(DEV)
    x = _kv(N * L, H, D, BF, 1).to(DEV)
    lens = torch.full((N,), L, dtype=I32, device=DEV)
    k, v = x[:, :H * D], x[:, H * D:2 * H * D]
    g.lfm2sc_cache8_write(k, v, *c.args, table, lens)
    ko, vo = g.lfm2sc_cache8_read(*c.args, table, lens, torch.empty(N * L, H * D, dtype=BF, device=DEV),
                                  torch.empty(N * L, H * D, dtype=BF, device=DEV))
    # e4m3 with a power-of-two scale: half a step of 2^-3, or of the smallest normal code's step below it
    for a, b in ((k, ko), (v, vo)):
        top = float(a.float().abs().max())
        assert ((a.double() - b.double()).abs() <= torch.maximum(a.double().abs() * 2.0 ** -4, torch.tensor(top * 2.0 ** -17, device=DEV))).all()


# ---------------------------------------------------------------- attention
def _attend(c, q, prefix_pages, prefix, table, lens, L, out_pad=8, **kw):
    P, H, S, D, B = c.shape
    N, W = table.shape[0], q.shape[1]
    out = torch.full((N * L + 1, W + out_pad), float("nan"), dtype=BF, device=DEV)
    bound = kw.get("max_suffix_len")
    n = g.lfm2sc_attn_cached8_workspace_bytes(BF, D, W // D, H, N, L, prefix, table.shape[1] * S if bound is None else bound)
    ws = torch.full((max(16, n),), 0xff, dtype=torch.uint8, device=DEV)
    g.lfm2sc_attn_cached8(q.to(DEV), *c.args, None if prefix_pages is None else torch.from_numpy(prefix_pages).to(DEV), prefix,
                          torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=I32, device=DEV), L, out[:N * L, :W], ws, **kw)
    assert torch.isnan(out[N * L:].float()).all() and torch.isnan(out[:, W:].float()).all()
    return out[:N * L, :W]


def _close(got, want, what=""):
    out, spread, most = want
    D = 128
    tol = HALF * (spread + 2 * np.abs(out)) * (1 + 2.0 ** -7) + (D + 10) * 2.0 ** -23 * (1 + most) * spread + 1e-30
    got = got.detach().cpu().double().numpy()
    bad = ~(np.abs(got - out) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} out of tolerance, first at {np.argwhere(bad)[0]}: {got[bad][0]} for "
                           f"{out[bad][0]} +- {tol[bad][0]}")


ATTEND = [
    # lens, L, prefix, S, B, Hq, Hkv, D
    ([1], 1, 0, 16, 16, 4, 1, 64),
    ([37], 1, 500, 16, 16, 32, 8, 64),
    ([64], 1, 0, 64, 64, 8, 8, 128),
    ([5, 0, 65, 128, 127], 1, 0, 16, 1, 8, 2, 64),
    ([5, 0, 65, 128, 127], 1, 63, 32, 16, 8, 2, 128),
    ([8, 3, 0, 100, 71], 8, 129, 64, 32, 20, 4, 128),
    ([8, 3, 0, 100, 71], 8, 0, 16, 16, 24, 2, 64),
    ([9, 400], 5, 1, 128, 128, 9, 3, 128),
    ([700, 33, 1500], 1, 0, 256, 1, 12, 1, 64),
    ([700, 33, 1500], 3, 2000, 16, 16, 32, 8, 64),
    ([20] * 40, 2, 130, 16, 16, 40, 8, 128),
    ([3000, 2999], 1, 0, 64, 16, 16, 2, 128),
    ([0, 0], 2, 0, 16, 16, 4, 2, 64),
    ([30], 40, 100, 32, 1, 6, 2, 64),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,L,prefix,S,B,Hq,Hkv,D", ATTEND)
def test_attention(lens, L, prefix, S, B, Hq, Hkv, D, fmt):
    N, most = len(lens), max(1, -(-max(lens) // S)) + 2
    npre = -(-prefix // S)
    P = npre + N * most
    c = Cache(fmt, P, Hkv, S, D, B, seed=L + prefix)
    order = np.random.default_rng(1).permutation(P).astype(np.int32)
    table = order[npre:].reshape(N, most).copy()
    for i, n in enumerate(lens):
        table[i, -(-n // S):] = 0x7fffffff                   # entries past a sequence's pages may hold anything
    gen = torch.Generator().manual_seed(4)
    q = torch.randn(N * L, Hq * D + 8, generator=gen).to(BF)[:, :Hq * D]
    want = o8.attention(q, c.host, order[:npre], prefix, table, lens, L, D ** -0.5)
    got = _attend(c, q, order[:npre] if npre else None, prefix, table, lens, L)
    _close(got, want, "table's width")
    again = _attend(c, q, order[:npre] if npre else None, prefix, table, lens, L)
    assert torch.equal(got, again)
    _close(_attend(c, q, order[:npre] if npre else None, prefix, table, lens, L, max_suffix_len=max(lens)), want, "bounded")


@pytest.mark.parametrize("fmt,B", [("int8", 1), ("e4m3", 1), ("e4m3", 16), ("int8", 16)])
def test_attention_ignores_what_lies_behind_a_sequence(fmt, B):
    """NaN codes and scales from a sequence's length on, in its own tile and pages."""
    lens, L, S, H, D = [1, 15, 16, 17, 40, 63, 70], 2, 32, 2, 64
    N, most = len(lens), 3
    c = Cache(fmt, N * most, H, S, D, B, seed=9)
    table = _table(N, most, N * most)
    q = torch.randn(N * L, 4 * D, generator=torch.Generator().manual_seed(1)).to(BF)
    want = o8.attention(q, c.host, None, 0, table, lens, L, D ** -0.5)
    k, v, ks, vs = c.args
    for i, n in enumerate(lens):
        for t in range(n, most * S):
            page = int(table[i, t // S])
            if fmt == "e4m3":
                k.view(torch.int8)[page, :, t % S] = 0x7f
                v.view(torch.int8)[page, :, t % S // 16, :, t % 16] = 0x7f
            if t % B == 0:
                ks[page, :, t % S // B] = float("nan")
                vs[page, :, t % S // B] = float("inf")
    _close(_attend(c, q, None, 0, table, lens, L), want)


def test_attention_bad_page_numbers_read_as_the_nearest():
    lens, L, S, H, D, B = [40, 33], 1, 16, 2, 64, 16
    c = Cache("e4m3", 4, H, S, D, B, seed=2)
    table = np.array([[-5, 2, 77], [1 << 30, 0, -(1 << 31)]], dtype=np.int32)
    prefix_pages = np.array([9, -1], dtype=np.int32)
    q = torch.randn(2, 4 * D, generator=torch.Generator().manual_seed(1)).to(BF)
    _close(_attend(c, q, prefix_pages, 20, table, lens, L), o8.attention(q, c.host, prefix_pages, 20, table, lens, L, D ** -0.5))


def test_attention_lengths_are_clamped():
    S, H, D, B = 16, 1, 64, 16
    c = Cache("int8", 4, H, S, D, B, seed=2)
    table = np.arange(4, dtype=np.int32).reshape(2, 2)
    q = torch.randn(2, D, generator=torch.Generator().manual_seed(1)).to(BF)
    _close(_attend(c, q, None, 0, table, [1 << 30, -7], 1), o8.attention(q, c.host, None, 0, table, [32, 0], 1, D ** -0.5))
    _close(_attend(c, q, None, 0, table, [25, 9], 1, max_suffix_len=20), o8.attention(q, c.host, None, 0, table, [20, 9], 1, D ** -0.5))


def test_attention_zero_scales_and_large_scores():
    """A head whose keys are all zeros (scale 0), and scores of some hundreds."""
    lens, S, H, D, B = [100, 64], 16, 2, 64, 16
    c = Cache("int8", 14, H, S, D, B, seed=6)
    c.args[2][:, 0] = 0.0
    c.args[2][:, 1] *= 40
    c.host = c.read()
    table = np.arange(14, dtype=np.int32).reshape(2, 7)
    q = torch.randn(2, 4 * D, generator=torch.Generator().manual_seed(1)).to(BF)
    _close(_attend(c, q, None, 0, table, lens, 1), o8.attention(q, c.host, None, 0, table, lens, 1, D ** -0.5))


def test_pool_past_32_bits():
    """Pages whose bytes lie past 2^32: written, read back and attended to."""
    H, S, D, B = 8, 128, 128, 16
    page = H * S * D
    P = (1 << 32) // page + 40
    k = torch.zeros(P, H, S, D, dtype=torch.int8, device=DEV)
    v = torch.zeros(P, H, S // 16, D, 16, dtype=torch.int8, device=DEV)
    ks, vs = torch.zeros(P, H, S // B, device=DEV), torch.zeros(P, H, S // B, device=DEV)
    T = 300
    table = torch.tensor([[P - 1, 7, P - 30]], dtype=I32, device=DEV)
    x = _kv(T, H, D, BF, 1).to(DEV)
    lens = torch.tensor([T], dtype=I32, device=DEV)
    g.lfm2sc_cache8_write(x[:, :H * D], x[:, H * D:2 * H * D], k, v, ks, vs, table, lens)
    small = (k[table[0].long()], v[table[0].long()], ks[table[0].long()], vs[table[0].long()])
    k2, v2, ks2, vs2 = (t.clone().zero_() for t in small)
    table2 = torch.arange(3, dtype=I32, device=DEV)[None]
    g.lfm2sc_cache8_write(x[:, :H * D], x[:, H * D:2 * H * D], k2, v2, ks2, vs2, table2, lens)
    for a, b in zip(small, (k2, v2, ks2, vs2)):
        assert torch.equal(a, b)
    out = [torch.empty(T, H * D, dtype=BF, device=DEV) for _ in range(4)]
    g.lfm2sc_cache8_read(k, v, ks, vs, table, lens, out[0], out[1])
    g.lfm2sc_cache8_read(k2, v2, ks2, vs2, table2, lens, out[2], out[3])
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])
    q = torch.randn(1, 16 * D, device=DEV).to(BF)
    got = []
    for cache, t in (((k, v, ks, vs), table), ((k2, v2, ks2, vs2), table2)):
        ws = torch.empty(max(16, g.lfm2sc_attn_cached8_workspace_bytes(BF, D, 16, H, 1, 1, 0, 384)), dtype=torch.uint8, device=DEV)
        got.append(g.lfm2sc_attn_cached8(q, *cache, None, 0, t, lens, 1, torch.empty_like(q), ws))
    assert torch.equal(got[0], got[1]) and bool(torch.isfinite(got[0]).all())
