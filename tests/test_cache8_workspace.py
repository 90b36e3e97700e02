"""Workspace sizes of the attention over the 8-bit cache (CPU): a workspace for the largest of a program's calls serves every
smaller one.  The splits of a call come from the library's plan itself."""
import ctypes
import itertools
import random

import pytest

from gated_short_causal_amd import _lib


class Plan(ctypes.Structure):
    _fields_ = [("form", ctypes.c_int), ("prefix_splits", ctypes.c_int), ("prefix_chunk", ctypes.c_int), ("suffix_splits", ctypes.c_int),
                ("prefix_blocks", ctypes.c_int64), ("suffix_blocks", ctypes.c_int64)]


DIRECT, SPLIT, SHARED = range(3)


def plan(D, Hq, Hkv, N, L, prefix, longest):
    f = getattr(_lib.hybrid_lib(), "_ZN6lfm2sc12cached8_planEiiiiiii")
    f.restype, f.argtypes = Plan, [ctypes.c_int] * 7
    return f(D, Hq, Hkv, N, L, prefix, longest)


def need(D, Hq, Hkv, N, L, prefix, longest):
    """What the launch writes: a row of D and a pair for each part of a row, where there is more than one."""
    p = plan(D, Hq, Hkv, N, L, prefix, longest)
    parts = p.prefix_splits + p.suffix_splits
    rows = N * L * Hq * parts if parts > 1 else 0
    return (rows * D * 4 + 255) // 256 * 256 + (rows * 8 + 255) // 256 * 256


HEADS = [(64, 32, 8), (128, 40, 8), (128, 24, 8), (64, 12, 1), (64, 16, 16), (128, 9, 3)]


def size(D, Hq, Hkv, *call):
    return _lib.hybrid_lib().lfm2sc_attn_cached8_workspace_bytes(0, D, Hq, Hkv, *call)


@pytest.mark.parametrize("heads", HEADS)
def test_a_larger_call_needs_no_less(heads):
    axes = ((1, 2, 3, 7, 16, 33, 63, 64, 65, 103, 128, 256, 257, 600, 2000), (1, 2, 5, 8, 64, 200),
            (0, 1, 64, 500, 1024, 4096, 8191, 20000, 65536), (0, 1, 37, 256, 257, 600, 1728, 1792, 2048, 4096, 20000))
    got = {}
    for at in itertools.product(*(range(len(a)) for a in axes)):
        call = tuple(a[i] for a, i in zip(axes, at))
        got[at] = size(*heads, *call)
        assert got[at] >= need(*heads, *call), call
        for axis in range(4):
            if at[axis]:
                below = got[at[:axis] + (at[axis] - 1,) + at[axis + 1:]]
                assert below <= got[at], (call, axis, below, got[at])


def test_random_calls_below_a_larger_one():
    rng = random.Random(5)

    def log(lo, hi):
        return min(hi, int(lo * (hi / lo) ** rng.random()))

    for _ in range(20000):
        heads = rng.choice(HEADS)
        N, L, prefix, longest = log(1, 5000), log(1, 300), rng.choice((0, log(1, 200000))), rng.choice((0, log(1, 200000)))
        most = size(*heads, N, L, prefix, longest)
        for call in ((N, L, prefix, longest), (rng.randint(1, N), L, prefix, longest), (N, L, prefix, rng.randint(0, longest)),
                     (rng.randint(1, N), rng.randint(1, L), rng.randint(0, prefix), rng.randint(0, longest))):
            assert need(*heads, *call) <= size(*heads, *call) <= most, (heads, N, L, prefix, longest, call)


def test_the_largest_sizes():
    """Sizes are computed in 64 bits, and stay within a few parts of the rows."""
    for N, L in (((1 << 28) // 32 - 1, 1), (1, (1 << 28) // 32 - 1), (1 << 10, 1 << 12)):
        for prefix, longest in itertools.product((0, 1, (1 << 30) - 1), repeat=2):
            got = size(64, 32, 8, N, L, prefix, longest)
            assert need(64, 32, 8, N, L, prefix, longest) <= got <= 2 * N * L * 32 * 264 + 512


def test_few_keys_need_none():
    for heads in HEADS:
        assert size(*heads, 1, 1, 500, 500) == 0 and size(*heads, 8, 1, 0, 256) == 0
        assert size(*heads, 10000, 1, 0, 256) == 0 and plan(*heads, 10000, 1, 0, 256).suffix_splits == 1


@pytest.mark.parametrize("kw,code", [(dict(plen=20000, N=3), 5), (dict(plen=4096, N=200, most=32, max=512), 5), (dict(most=256, max=4096), 5)])
def test_a_smaller_workspace_is_refused(kw, code):
    from test_cache8_abi import ATT
    args = {**ATT, **kw}
    args["wsb"] = size(64, 8, 2, args["N"], args["L"], args["plen"], args["max"]) - 1
    assert _lib.hybrid_lib().lfm2sc_attn_cached8(*args.values()) == code
