"""Writes into the 8-bit cache that the header's small print is about (GPU), against the oracle bit for bit."""
import numpy as np
import pytest
import torch

from oracle import cache8 as o8
from test_gpu_cache8 import BF, F32, Cache, _kv, _write

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("D,S,B", [(64, 16, 16), (128, 64, 64)])
@pytest.mark.parametrize("old", [0.0, 2.0 ** -101, NAN, INF, -1.0, 2.0 ** -60])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_a_block_whose_old_scale_is_no_use(fmt, old, D, S, B):
    """Rows join a block with a scale of 0, too small, not finite, negative, or 2^40 times too small for them: a new scale, zeros
    of the earlier codes, and an earlier NaN code (e4m3) stays NaN."""
    H, held, n = 2, 5, 3
    c = Cache(fmt, 2, H, S, D, B)
    for scales in c.args[2:]:
        scales.fill_(old)
    if fmt == "e4m3":
        c.args[0].view(torch.int8)[:, :, 2] = 0x7f           # token 2 of k, and of v
        c.args[1].view(torch.int8)[:, :, 0, :, 2] = 0x7f
    c.host = c.read()
    _write(c, _kv(n, H, D, BF, 1), np.array([[1]], dtype=np.int32), [held + n], [n])
    c.check()
    got = c.read()
    for codes, scales in (("k", "ks"), ("v", "vs")):
        kept = got[codes][1, :, :held]
        assert np.isnan(kept[:, 2]).all() == (fmt == "e4m3") and (np.delete(kept, 2, 1) == 0).all()
        assert (got[scales][1, :, 0] > 2.0 ** -20).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B", [1, 16])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_infinities_where_nothing_is_finite(fmt, B, dtype):
    """A scale of 0, as for zeros, and codes of NaN (e4m3) or 0 (int8); beside a finite value, the largest code."""
    H, D, S = 1, 64, 16
    c = Cache(fmt, 1, H, S, D, B)
    x = torch.zeros(2 * S, 2 * D, dtype=dtype)[:S]
    x[3, 7], x[3, 9], x[3, D + 8] = INF, -INF, INF
    if B == 1:
        x[5, 1], x[5, 2], x[5, D + 1], x[5, D + 2] = INF, 2.0, -INF, -3.0
    _write(c, x, np.array([[0]], dtype=np.int32), [S], [S])
    c.check()
    got = c.read()
    for code in (got["k"][0, 0, 3, 7], got["k"][0, 0, 3, 9], got["v"][0, 0, 3, 8]):
        assert np.isnan(code) if fmt == "e4m3" else code == 0
    assert got["ks"][0, 0, 3 // B] == 0 and got["vs"][0, 0, 3 // B] == 0
    if B == 1:
        top = 448 if fmt == "e4m3" else 127
        assert got["k"][0, 0, 5, 1] == top and got["v"][0, 0, 5, 1] == -top


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_taken_back_leave_their_scale(fmt):
    """A large draft that is taken back: its block's scale stays, and the earlier values stay within one step of it."""
    H, D, S, B, held = 2, 64, 16, 16, 6
    c = Cache(fmt, 1, H, S, D, B, full=False)
    table, x = np.array([[0]], dtype=np.int32), _kv(held, H, D, BF, 1)
    _write(c, x, table, [held], [held])
    first = c.read()
    _write(c, _kv(4, H, D, BF, 2, amp=1000.0), table, [held + 4], [4])
    marked = c.read()
    assert (marked["ks"] > first["ks"]).all()
    _write(c, _kv(1, H, D, BF, 3), table, [held + 1], [1])   # the drafts are taken back
    c.check()
    got = c.read()
    assert (got["ks"] == marked["ks"]).all() and (got["vs"] == marked["vs"]).all()
    k, _ = o8.values(c.host, [0], held)
    # one step of the scale: 1 for int8, 2^-3 of the value or the smallest codes' 2^-9 for e4m3
    off = np.abs(k.reshape(held, -1) - x[:, :H * D].double().numpy())
    step = np.repeat(got["ks"][0, :, 0].astype(np.float64), D)
    value = np.abs(x[:, :H * D].double().numpy())
    assert (off <= (step if fmt == "int8" else np.maximum(value / 8, step * 2.0 ** -9))).all()
