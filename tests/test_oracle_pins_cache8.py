"""Pins of oracle/cache8.py: hand-worked codes and scales, rotary positions as complex numbers, and attention over a cache of
unit scales against the bf16 cache's oracle formula (CPU)."""
import numpy as np
import pytest
import torch

from oracle import cache8 as o8


def test_codes_by_hand():
    x = np.array([0.0, 0.49, 0.5, 1.5, -2.5, 126.6, 127.4, 200.0, -np.inf, np.nan])
    assert o8.round_code(x, True).tolist() == [0, 0, 0, 2, -2, 127, 127, 127, -127, 0]
    # e4m3: steps of 2^-9 below 2^-6, then an eighth of the power of two; 17 lies between 16 and 18, 19 between 18 and 20
    x = np.array([0.0, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 440.0, 500.0, -np.inf])
    assert o8.round_code(x, False).tolist() == [0, 0, 2.0 ** -8, 16, 20, 448, 448, -448]
    assert np.isnan(o8.round_code(np.array([np.nan]), False)).all()


def test_codes_are_torchs_float8():
    x = torch.linspace(-448, 448, 100001).float()
    x = torch.cat([x, x * 2.0 ** -12, torch.randn(10000, generator=torch.Generator().manual_seed(0))])
    assert (o8.round_code(x.numpy(), False) == x.to(torch.float8_e4m3fn).double().numpy()).all()


@pytest.mark.parametrize("top,int8,scale", [
    (254.0, True, 2.0), (0.0, True, 0.0), (1e-38, True, 2.0 ** -100), (448.0, False, 1.0), (449.0, False, 2.0), (224.0, False, 0.5),
    (225.0, False, 1.0), (1.0, False, 2.0 ** -8), (0.0, False, 0.0), (1e-38, False, 2.0 ** -100), (3e38, False, 2.0 ** 120)])
def test_fresh_scales(top, int8, scale):
    got = o8.fresh(np.float32(top), int8)
    assert got.dtype == np.float32 and got == np.float32(scale)


def test_joined_scales():
    assert o8.joined(np.float32(2.0), 100.0, True) == (2.0, 1.0)
    assert o8.joined(np.float32(2.0), 254.9, True) == (2.0, 1.0)          # 127.45 rounds to 127
    assert o8.joined(np.float32(2.0), 255.0, True) == (4.0, 0.5)
    assert o8.joined(np.float32(2.0), 1020.0, True) == (16.0, 0.125)      # 510 = 4 x 127.5 does not fit 8
    assert o8.joined(np.float32(0.5), 224.0, False) == (0.5, 1.0)
    assert o8.joined(np.float32(0.5), 225.0, False) == (1.0, 0.5)
    assert o8.joined(np.float32(0.0), 127.0, True) == (1.0, 0.0)
    assert o8.joined(np.float32(np.nan), 127.0, True) == (1.0, 0.0)
    assert o8.joined(np.float32(2.0 ** -90), 127.0, True) == (1.0, 0.0)  # 2^90 times too small


def _cache(int8, P, H, S, D, B):
    return {"page": S, "block": B, "int8": int8, "k": np.zeros((P, H, S, D)), "v": np.zeros((P, H, S, D)),
            "ks": np.zeros((P, H, S // B), np.float32), "vs": np.zeros((P, H, S // B), np.float32)}


def test_write_by_hand():
    c = _cache(True, 2, 1, 16, 2, 16)
    table = np.array([[1]], dtype=np.int32)
    o8.write(c, np.array([[127.0, 3.4]]), np.array([[0.0, -254.0]]), table, [1], [1])
    assert c["k"][1, 0, 0].tolist() == [127, 3] and c["ks"][1, 0, 0] == 1.0
    assert c["v"][1, 0, 0].tolist() == [0, -127] and c["vs"][1, 0, 0] == 2.0 and c["ks"][0, 0, 0] == 0.0
    o8.write(c, np.array([[300.0, 0.0], [4.0, -6.0]]), np.array([[10.0, 3.0], [1.0, 0.0]]), table, [3], [2])
    assert c["ks"][1, 0, 0] == 4.0 and c["k"][1, 0, :3].tolist() == [[32, 1], [75, 0], [1, -2]]
    assert c["vs"][1, 0, 0] == 2.0 and c["v"][1, 0, :3].tolist() == [[0, -127], [5, 2], [0, 0]]
    k, v = o8.values(c, [1], 3)
    assert k[:, 0].tolist() == [[128, 4], [300, 0], [4, -8]] and v[1, 0].tolist() == [10, 4]


def test_rotary_is_a_complex_product():
    gen = torch.Generator().manual_seed(0)
    x, f = torch.randn(5, 2 * 16, generator=gen).double(), torch.rand(3, generator=gen).double()
    pos = np.array([0, 1, 7, -2, 1000])
    y = o8.rotary(x, 16, f, pos, interleaved=True, magnitude=2.0)
    z = torch.view_as_complex(x.reshape(5, 2, 8, 2)[:, :, :3].contiguous())
    w = z * torch.polar(torch.full((5, 1, 3), 2.0).double(), torch.from_numpy(pos).double()[:, None, None] * f)
    assert np.allclose(y.reshape(5, 2, 16)[:, :, :6], torch.view_as_real(w).reshape(5, 2, 6).numpy(), rtol=0, atol=1e-12)
    assert (y.reshape(5, 2, 16)[:, :, 6:] == x.reshape(5, 2, 16)[:, :, 6:].numpy()).all()
    order = [0, 3, 1, 4, 2, 5] + list(range(6, 16))          # interleaved columns of a half layout
    half = x.reshape(5, 2, 16)
    inter = torch.empty_like(half)
    inter[:, :, :] = half[:, :, order]
    a = o8.rotary(half.reshape(5, 32), 16, f, pos).reshape(5, 2, 16)[:, :, order]
    b = o8.rotary(inter.reshape(5, 32), 16, f, pos, interleaved=True).reshape(5, 2, 16)
    assert np.allclose(a, b, rtol=0, atol=1e-13)
    back = o8.rotary(o8.rotary(x, 16, f, pos, magnitude=2.0), 16, f, pos, inverse=True, magnitude=0.5)
    assert np.allclose(back, x.numpy(), rtol=0, atol=1e-12)


def test_attention_by_torch():
    gen = torch.Generator().manual_seed(1)
    c = _cache(True, 6, 2, 16, 8, 16)
    c["k"][:], c["v"][:] = (torch.randint(-127, 128, (6, 2, 16, 8), generator=gen).numpy() for _ in range(2))
    c["ks"][:], c["vs"][:] = (torch.rand(6, 2, 1, generator=gen).numpy() * 0.02 for _ in range(2))
    q = torch.randn(4, 4 * 8, generator=gen).double()
    table, lens = np.array([[2, 5], [0, 1]], dtype=np.int32), [20, 1]
    out, _, _ = o8.attention(q, c, [4, 3], 18, table, lens, 2, 0.3)
    dense = torch.from_numpy(c["k"] * c["ks"][..., None]), torch.from_numpy(c["v"] * c["vs"][..., None])
    for i in range(2):
        ks, vs = (torch.cat([x[[4, 3]].transpose(1, 2).reshape(32, 2, 8)[:18], x[table[i]].transpose(1, 2).reshape(32, 2, 8)[:lens[i]]])
                  for x in dense)
        for s in range(2):
            n = 18 + max(0, lens[i] - 1 + s)
            for h in range(4):
                p = torch.softmax(0.3 * ks[:n, h // 2] @ q[2 * i + s, 8 * h:8 * h + 8], 0)
                assert np.allclose(out[2 * i + s, 8 * h:8 * h + 8], (p @ vs[:n, h // 2]).numpy(), rtol=0, atol=1e-12)
