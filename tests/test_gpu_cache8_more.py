"""The rotary positions and the 8-bit cache in use (GPU): written, grown and attended to step by step, captured, on several
streams, with every form of the attention, and with device data at its limits.  Tolerances as in test_gpu_cache8."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import gated_short_causal_amd as g
from oracle import cache8 as o8
from test_gpu_cache8 import BF, DEV, F32, I32, Cache, _attend, _close, _kv, _table, _write

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("fmt,S,B,D", [("e4m3", 16, 16, 64), ("int8", 64, 32, 128), ("int8", 32, 1, 64), ("e4m3", 128, 128, 128)])
def test_decode_and_verify_over_a_shared_prefix(fmt, S, B, D):
    """Prefix and prompts written packed, decode steps, verify blocks of which a part is taken back and written again."""
    Hq, Hkv, N, prefix = 8, 2, 3, 75
    prompts, limit = [20, 1, 90], 160
    most, npre = -(-limit // S), -(-prefix // S)
    P = npre + N * most
    c = Cache(fmt, P, Hkv, S, D, B, full=False)
    order = np.random.default_rng(3).permutation(P).astype(np.int32)
    pp, table = order[:npre], order[npre:].reshape(N, most)
    _write(c, _kv(prefix, Hkv, D, BF, 1), pp[None], [prefix], [prefix])
    _write(c, _kv(sum(prompts), Hkv, D, BF, 2), table, prompts, prompts)
    c.check("prompts")
    freqs, lens = g.lfm2sc_rotary_freqs(D).to(DEV), list(prompts)
    for step, (L, back) in enumerate([(1, 0), (1, 0), (6, 4), (6, 5), (1, 0), (8, 0)]):
        lens = [n + L for n in lens]
        gen = torch.Generator().manual_seed(10 + step)
        rows = torch.randn(N * L, (Hq + 2 * Hkv) * D, generator=gen).to(BF).to(DEV)
        q, kv = rows[:, :Hq * D], rows[:, Hq * D:]
        pos = torch.tensor([prefix + n - L + s for n in lens for s in range(L)], dtype=I32, device=DEV)
        plain = rows.cpu()
        g.lfm2sc_rotary(q, q, D, freqs, positions=pos, k=kv[:, :Hkv * D], k_out=kv[:, :Hkv * D])
        turned = o8.rotary(plain[:, :(Hq + Hkv) * D], D, freqs.cpu(), pos.cpu().numpy())
        assert np.abs(rows[:, :(Hq + Hkv) * D].cpu().double().numpy() - turned).max() <= np.abs(turned).max() * 2.0 ** -8
        assert torch.equal(rows[:, (Hq + Hkv) * D:].cpu(), plain[:, (Hq + Hkv) * D:])
        _write(c, kv.cpu(), table, lens, [L] * N, uniform=True)
        c.check(f"step {step}")
        got = _attend(c, q.cpu(), pp, prefix, table, lens, L, max_suffix_len=limit)
        _close(got, o8.attention(q.cpu(), c.host, pp, prefix, table, lens, L, D ** -0.5), f"step {step}")
        lens = [n - back for n in lens]


@pytest.mark.parametrize("fmt,B", [("e4m3", 16), ("e4m3", 1), ("int8", 16), ("int8", 1)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,L,G,prefix,S", [(33, 1, 4, 63, 16), (9, 8, 2, 64, 32), (16, 3, 3, 65, 64), (43, 3, 1, 130, 16),
                                            (64, 2, 2, 250, 128), (129, 1, 1, 1, 16), (5, 9, 5, 450, 16)])
def test_shared_prefix_of_many_rows(N, L, G, prefix, S, D, fmt, B):
    """More than 128 rows a key/value head: the prefix of one to eight tiles, rows that fill their last block or one row of
    it; codes and scales behind the prefix's end are NaN."""
    Hkv, lens = 2, [(7 * i) % 40 + L for i in range(N)]
    lens[0], lens[1] = 0, L - 1
    most, npre = -(-max(lens) // S), -(-prefix // S)
    P = npre + N * most
    c = Cache(fmt, P, Hkv, S, D, B, seed=N)
    order = np.random.default_rng(N).permutation(P).astype(np.int32)
    pp, table = order[:npre], order[npre:].reshape(N, most)
    q = torch.randn(N * L, Hkv * G * D, generator=torch.Generator().manual_seed(1)).to(BF)
    want = o8.attention(q, c.host, pp, prefix, table, lens, L, D ** -0.5)
    k, v, ks, vs = c.args
    for t in range(prefix, npre * S):
        page = int(pp[t // S])
        if fmt == "e4m3":
            k.view(torch.int8)[page, :, t % S] = 0x7f
            v.view(torch.int8)[page, :, t % S // 16, :, t % 16] = 0x7f
        if t % B == 0:
            ks[page, :, t % S // B] = float("nan")
            vs[page, :, t % S // B] = float("nan")
    got = _attend(c, q, pp, prefix, table, lens, L)
    _close(got, want)
    assert torch.equal(got, _attend(c, q, pp, prefix, table, lens, L))


@pytest.mark.parametrize("N,L,prefix,S,own", [(2, 1, 100, 32, 30), (3, 2, 2000, 16, 17), (70, 1, 70, 16, 20), (1, 20, 1100, 64, 700)])
@pytest.mark.parametrize("B", [1, 16])
def test_prefix_end_inside_a_tile(N, L, prefix, S, own, B):
    """The other forms (few rows): one launch for few keys, and splits joined."""
    Hkv, G, D = 2, 2, 64
    lens = [own] * N
    most, npre = -(-own // S), -(-prefix // S)
    P = npre + N * most
    c = Cache("e4m3", P, Hkv, S, D, B, seed=N)
    pp, table = np.arange(npre, dtype=np.int32), np.arange(npre, P, dtype=np.int32).reshape(N, most)
    q = torch.randn(N * L, Hkv * G * D, generator=torch.Generator().manual_seed(1)).to(BF)
    want = o8.attention(q, c.host, pp, prefix, table, lens, L, D ** -0.5)
    k, v, ks, vs = c.args
    tail = prefix % S
    if tail:
        k.view(torch.int8)[npre - 1, :, tail:] = 0x7f
        for t in range(tail, S):
            v.view(torch.int8)[npre - 1, :, t // 16, :, t % 16] = 0x7f
        ks[npre - 1, :, -(-tail // B):] = float("nan")
        vs[npre - 1, :, -(-tail // B):] = float("inf")
    _close(_attend(c, q, pp, prefix, table, lens, L), want)


def test_many_sequences():
    """More sequences than the one-trip search holds, some empty, in every call that packs rows."""
    N, H, S, D, B = 700, 1, 16, 64, 16
    lens = [(i * 7) % 5 for i in range(N)]
    held = [(i * 3) % 11 for i in range(N)]
    c = Cache("e4m3", N + 1, H, S, D, B, seed=1)
    table = _table(N, 1, N + 1)
    ends = [a + b for a, b in zip(held, lens)]
    _write(c, _kv(sum(lens), H, D, BF, 2), table, ends, lens, lead=3, tail=2)
    c.check()
    cu = torch.tensor([3] + lens).cumsum(0).to(I32)
    T = int(cu[-1]) + 2
    out = torch.full((T, 2 * D), float("nan"), dtype=F32, device=DEV)
    g.lfm2sc_cache8_read(*c.args, torch.from_numpy(table).to(DEV), torch.tensor(ends, dtype=I32, device=DEV), out[:, :D], out[:, D:],
                         cu_seqlens=cu.to(DEV))
    got = out.cpu().double().numpy()
    assert np.isnan(got[:3]).all() and np.isnan(got[T - 2:]).all()
    for i in range(N):
        k, v = o8.values(c.host, table[i], ends[i]) if ends[i] else (np.zeros((0, 1, D)),) * 2
        rows = np.concatenate([k[:, 0], v[:, 0]], 1)[ends[i] - lens[i]:]
        assert (got[cu[i]:cu[i + 1]] == rows.astype(np.float32)).all(), i
    x = _kv(T, 1, D, F32, 5)[:, :D].contiguous()
    starts = torch.arange(N, dtype=I32) * 5
    y = torch.full((T, D), float("nan"), device=DEV)
    freqs = g.lfm2sc_rotary_freqs(D)
    g.lfm2sc_rotary(x.to(DEV), y, D, freqs.to(DEV), positions=starts.to(DEV), cu_seqlens=cu.to(DEV))
    pos, mine = o8.packed_positions(cu.tolist(), T, starts.tolist())
    want = o8.rotary(x, D, freqs, pos)
    got = y.cpu().double().numpy()
    assert np.isnan(got[~mine]).all()
    # a pair's magnitudes are at most twice its larger result's scale
    assert (np.abs(got - want)[mine] <= 2.0 ** -20 * np.abs(x.double().numpy()[mine]).max(1, keepdims=True)).all()


def _setup(fmt="int8", N=4, L=2, D=64, Hq=8, Hkv=2, S=16, B=16, prefix=200, limit=64, seed=0):
    npre, most = -(-prefix // S), -(-limit // S)
    P = npre + N * most
    c = Cache(fmt, P, Hkv, S, D, B, seed=seed)
    pp = torch.arange(npre, dtype=I32, device=DEV)
    table = torch.arange(npre, P, dtype=I32, device=DEV).reshape(N, most)
    rows = torch.randn(N * L, (Hq + 2 * Hkv) * D, device=DEV).to(BF)
    lens = torch.tensor([10 + 5 * i for i in range(N)], dtype=I32, device=DEV)
    pos = torch.arange(N * L, dtype=I32, device=DEV)
    freqs = g.lfm2sc_rotary_freqs(D).to(DEV)
    out = torch.empty(N * L, Hq * D, dtype=BF, device=DEV)
    ws = torch.empty(max(16, g.lfm2sc_attn_cached8_workspace_bytes(BF, D, Hq, Hkv, N, L, prefix, limit)), dtype=torch.uint8, device=DEV)
    turned = torch.empty(N * L, (Hq + Hkv) * D, dtype=BF, device=DEV)

    def step():
        q, k = turned[:, :Hq * D], turned[:, Hq * D:]
        g.lfm2sc_rotary(rows[:, :Hq * D], q, D, freqs, positions=pos, k=rows[:, Hq * D:(Hq + Hkv) * D], k_out=k)
        g.lfm2sc_cache8_write(k, rows[:, (Hq + Hkv) * D:], *c.args, table, lens)
        g.lfm2sc_attn_cached8(q, *c.args, pp, prefix, table, lens, L, out, ws)
    return c, rows, lens, pos, out, step


@pytest.mark.parametrize("N,prefix", [(4, 200), (4, 5000), (80, 300)])
def test_a_captured_step_replays(N, prefix):
    """Rotate, write and attend in one graph: lengths, positions and rows change between replays, the cache grows."""
    c, rows, lens, pos, out, step = _setup(N=N, prefix=prefix, limit=500)
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


def test_streams_side_by_side():
    """Two steps over caches and workspaces of their own, on two streams, each queued behind work of its stream."""
    steps = [_setup(seed=s, prefix=3000, N=40) for s in (1, 2)]
    want = []
    for c, rows, lens, pos, out, step in steps:
        codes, scales = c.codes.clone(), c.scales.clone()
        step()
        torch.cuda.synchronize()
        want.append((out.clone(), c.codes.clone()))
        c.codes.copy_(codes)
        c.scales.copy_(scales)
        out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    kept = [s[1].clone() for s in steps]
    for s in steps:
        s[1].zero_()
    torch.cuda.synchronize()
    for (c, rows, lens, pos, out, step), stream, x in zip(steps, streams, kept):
        with torch.cuda.stream(stream):
            rows.copy_(x)
            step()
    torch.cuda.synchronize()
    for s, (out, codes) in zip(steps, want):
        assert torch.equal(s[4], out) and torch.equal(s[0].codes, codes)


def test_a_nan_query_stays_in_its_row():
    c, rows, lens, pos, out, step = _setup(N=70, L=2, prefix=300)
    step()
    torch.cuda.synchronize()
    before = out.clone()
    rows[5, :64] = float("nan")                              # one head of one row's query
    step()
    torch.cuda.synchronize()
    assert torch.isnan(out[5, :64].float()).all()
    out[5, :64] = before[5, :64]
    assert torch.equal(out, before)


def test_calls_without_rows_or_keys():
    """Calls without rows, without sequences and without keys."""
    c, rows, lens, pos, out, step = _setup()
    k, none = rows[:0, :128], torch.empty(0, 4, dtype=I32, device=DEV)
    before = c.codes.clone()
    g.lfm2sc_cache8_write(k, k, *c.args, none, lens[:0])
    g.lfm2sc_cache8_write(k, k, *c.args, torch.zeros(4, 4, dtype=I32, device=DEV), lens, cu_seqlens=torch.zeros(5, dtype=I32, device=DEV))
    g.lfm2sc_rotary(k, k, 64, g.lfm2sc_rotary_freqs(64).to(DEV), positions=lens[:0])
    torch.cuda.synchronize()
    assert torch.equal(c.codes, before)
    q = torch.ones(600, 512, dtype=BF, device=DEV)
    o = torch.full_like(q, float("nan"))
    ws = torch.empty(16, dtype=torch.uint8, device=DEV)
    g.lfm2sc_attn_cached8(q, *c.args, None, 0, torch.empty(600, 0, dtype=I32, device=DEV), torch.zeros(600, dtype=I32, device=DEV), 1, o, ws)
    assert (o == 0).all()


_CHECK = """
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

k, v = (torch.zeros(8, 2, *s, dtype=torch.int8, device=d) for s in ((16, 64), (1, 64, 16)))
ks, vs = torch.ones(8, 2, 1, device=d), torch.ones(8, 2, 1, device=d)
x = torch.randn(6, 128, device=d).to(BF)
table = ints(1, 2, 3, -1).reshape(2, 2)
def write(lens, cu=None, t=table):
    return status(lambda: g.lfm2sc_cache8_write(x, x, k, v, ks, vs, t, lens, cu_seqlens=cu))
def read(lens, cu=None, t=table):
    return status(lambda: g.lfm2sc_cache8_read(k, v, ks, vs, t, lens, x, x, cu_seqlens=cu))
def attend(lens, pp=0, most=None):
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=d)
    return status(lambda: g.lfm2sc_attn_cached8(x[:2], k, v, ks, vs, ints(pp), 10, table, lens, 1, torch.empty_like(x[:2]), ws, max_suffix_len=most))
def rotate(*cu):
    return status(lambda: g.lfm2sc_rotary(x, torch.empty_like(x), 64, g.lfm2sc_rotary_freqs(64).to(d), cu_seqlens=ints(*cu)))
s = [write(ints(32, 16)), write(ints(32, 17)), write(ints(33, 16)), write(ints(3, 3), ints(0, 2, 6)), write(ints(3, 3), ints(0, 7, 6)),
     write(ints(3, 3), None, ints(8, 0, 0, 0).reshape(2, 2)), read(ints(32, 16)), read(ints(32, 17)), attend(ints(32, 16)), attend(ints(32, 17)),
     attend(ints(32, 16), 8), attend(ints(32, 16), 0, 31), rotate(0, 2, 6), rotate(3, 2)]
torch.cuda.synchronize()
print("STATUS", s)
"""


def test_check_mode():
    """LFM2SC_CHECK=1 (read once per process, hence a child): pages, lengths and row offsets out of range are
    LFM2SC_ERR_PRECONDITION (6); entries that no token uses may hold anything."""
    r = subprocess.run([sys.executable, "-c", _CHECK, ROOT], env=dict(os.environ, LFM2SC_CHECK="1"), capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    line = [x for x in r.stdout.splitlines() if x.startswith("STATUS")][0]
    assert line == "STATUS [0, 6, 6, 0, 6, 6, 0, 6, 0, 6, 6, 6, 0, 6]", line


def test_example_decodes():
    from examples import hybrid_step
    torch.manual_seed(0)
    for codes in (torch.float8_e4m3fn, torch.int8):
        r = hybrid_step.decode_8bit([20, 3], 3, 70, torch.device(DEV), codes=codes)
        assert r["out"].shape == (3, 2, 2048) and torch.isfinite(r["out"].float()).all() and r["lens"].tolist() == [23, 6]


@pytest.mark.parametrize("L", [1, 5, 16, 33])
@pytest.mark.parametrize("fmt,S,B", [("e4m3", 16, 16), ("int8", 64, 64), ("int8", 32, 1)])
def test_a_padded_batch(fmt, S, B, L):
    """Rows of every sequence, of which some hold fewer tokens than rows, or none: the rows before token 0 are left out, written
    and read."""
    H, D, lens = 2, 64, [0, 1, L, max(L - 2, 0), 3 * L + 7, 0]
    N, most = len(lens), -(-(3 * L + 7) // S)
    c = Cache(fmt, N * most, H, S, D, B, seed=L)
    table = _table(N, most, N * most)
    _write(c, _kv(N * L, H, D, BF, 3), table, lens, [L] * N, uniform=True)
    c.check()
    out = torch.full((N * L, 2 * H * D), float("nan"), dtype=F32, device=DEV)
    g.lfm2sc_cache8_read(*c.args, torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=I32, device=DEV), out[:, :H * D], out[:, H * D:])
    got = out.cpu().double().numpy().reshape(N, L, 2, H, D)
    for i, n in enumerate(lens):
        there = min(n, L)
        assert np.isnan(got[i, :L - there]).all(), i
        if there:
            k, v = o8.values(c.host, table[i], n)
            want = np.stack([k, v], 1)[n - there:].astype(np.float32)
            assert (got[i, L - there:] == want).all(), i


@pytest.mark.parametrize("N,L,G,prefix,own", [(1, 8, 32, 3000, 20), (1, 1, 64, 0, 700), (2, 70, 2, 900, 100), (3, 5, 16, 40, 9),
                                              (1, 1, 16, 5000, 0), (1, 200, 1, 64, 200), (40, 1, 64, 0, 300)])
@pytest.mark.parametrize("fmt,B", [("int8", 16), ("e4m3", 1)])
def test_wide_groups_and_long_blocks(N, L, G, prefix, own, fmt, B):
    """One key/value head for many query heads, blocks of more rows than a tile has, and a prefix with nothing behind it."""
    Hkv, D, S = 1, 64, 32
    most, npre = -(-max(own, 1) // S), -(-prefix // S)
    P = npre + N * most
    c = Cache(fmt, P, Hkv, S, D, B, seed=G)
    order = np.random.default_rng(1).permutation(P).astype(np.int32)
    pp, table, lens = order[:npre], order[npre:].reshape(N, most), [max(own - 3 * i, 0) for i in range(N)]
    q = torch.randn(N * L, Hkv * G * D, generator=torch.Generator().manual_seed(1)).to(BF)
    got = _attend(c, q, pp if npre else None, prefix, table, lens, L)
    _close(got, o8.attention(q, c.host, pp if npre else None, prefix, table, lens, L, D ** -0.5))


def test_page_numbers_used_by_two_sequences():
    """Sequences may read the same pages."""
    c = Cache("int8", 6, 2, 16, 64, 16)
    table, lens = np.array([[0, 1, 2], [0, 1, 3], [0, 1, 2]], dtype=np.int32), [40, 45, 40]
    q = torch.randn(3, 256, generator=torch.Generator().manual_seed(1)).to(BF)
    q[2] = q[0]
    got = _attend(c, q, None, 0, table, lens, 1)
    _close(got, o8.attention(q, c.host, None, 0, table, lens, 1, 64 ** -0.5))
    assert torch.equal(got[0], got[2])


@pytest.mark.parametrize("N,L,prefix,own", [(3, 2, 0, 21), (2, 3, 1500, 37), (70, 2, 100, 21)])
@pytest.mark.parametrize("B", [1, 16])
def test_a_tiny_scale(N, L, prefix, own, B):
    """Scores that underflow, of blocks of zeros among them, weigh alike, and keys past the end nothing: every form."""
    Hkv, G, D, S = 2, 2, 64, 32
    most, npre = -(-own // S), -(-prefix // S)
    P = npre + N * most
    c = Cache("int8", P, Hkv, S, D, B, seed=N)
    c.args[2][::2] = 0.
    c.host = c.read()
    pp, table = np.arange(npre, dtype=np.int32), np.arange(npre, P, dtype=np.int32).reshape(N, most)
    q = torch.randn(N * L, Hkv * G * D, generator=torch.Generator().manual_seed(1)).to(BF)
    for scale in (1e-12, 1e-38):
        got = _attend(c, q, pp if npre else None, prefix, table, [own] * N, L, scale=scale)
        _close(got, o8.attention(q, c.host, pp if npre else None, prefix, table, [own] * N, L, scale))
