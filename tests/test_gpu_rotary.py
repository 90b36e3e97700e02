"""lfm2sc_rotary on the GPU against the fp64 oracle.

Tolerance of a pair (x, y): cos and sin are polynomials in an fp32 argument of at most pi / 4 (its rounding 2^-25, the
evaluation's last operations 2 x 2^-24, the truncation 2^-28), times the magnitude (2^-24), two products and a sum in fp32
(2 x 2^-24): below 2^-21 m (|x| + |y|); the angle itself is off by 4 roundings of 2^-53 of it.  bf16 results are rounded
once more, half a step.
"""
import numpy as np
import pytest
import torch

import gated_short_causal_amd as g
from oracle import cache8 as o8

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _check(got, x, D, freqs, pos, rows=None, what="", **kw):
    m = kw.get("magnitude", 1.0)
    want = o8.rotary(x, D, freqs, pos, **kw)
    a = np.abs(o8.f64(x)).reshape(x.shape[0], -1, D)
    R = 2 * freqs.numel()
    pair = np.zeros_like(a)
    i, j = (np.arange(0, R, 2), np.arange(1, R, 2)) if kw.get("interleaved") else (np.arange(R // 2), np.arange(R // 2, R))
    angle = np.abs(np.asarray(pos, dtype=np.float64))[:, None] * o8.f64(freqs) * 2.0 ** -51
    pair[:, :, i] = pair[:, :, j] = abs(m) * (a[:, :, i] + a[:, :, j]) * (2.0 ** -21 + angle)[:, None]
    tol = pair.reshape(want.shape) + torch.finfo(x.dtype).eps / 2 * np.abs(want)
    tol += 1e-37
    got = got.detach().cpu().double().numpy()
    rows = np.ones(x.shape[0], dtype=bool) if rows is None else rows
    bad = ~(np.abs(got - want) <= tol) & rows[:, None]
    assert not bad.any(), f"{what}: {bad.sum()} off, first {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"
    stay = np.ones(D, dtype=bool)
    stay[:R] = False
    same = (got == o8.f64(x)).reshape(a.shape)[:, :, stay]
    assert same[rows].all(), what
    return got


def _rows(T, width, dtype, seed, pad=8):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(T, width + pad, generator=gen).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 32), (128, 128), (128, 2), (128, 126), (80, 80), (80, 40), (96, 68), (256, 256),
                                 (8, 8), (8, 2), (24, 10), (512, 512), (72, 72)])
def test_positions(D, R, interleaved, dtype):
    T, Hq, Hkv = 7, 3, 2
    base = _rows(T, (Hq + Hkv) * D, dtype, D + R)
    freqs = g.lfm2sc_rotary_freqs(R)
    pos = torch.tensor([0, 1, 2, 1000, 65535, 1 << 20, -5], dtype=I32)
    x = base.to(DEV)
    q, k = x[:, :Hq * D], x[:, Hq * D:(Hq + Hkv) * D]
    for inverse, magnitude in ((False, 1.0), (True, 1.25)):
        qo = torch.full((T, Hq * D + 16), float("nan"), dtype=dtype, device=DEV)
        ko = torch.full((T, Hkv * D), float("nan"), dtype=dtype, device=DEV)
        g.lfm2sc_rotary(q, qo[:, :Hq * D], D, freqs.to(DEV), positions=pos.to(DEV), k=k, k_out=ko, interleaved=interleaved,
                        inverse=inverse, magnitude=magnitude)
        kw = dict(interleaved=interleaved, inverse=inverse, magnitude=magnitude)
        _check(qo[:, :Hq * D], base[:, :Hq * D], D, freqs, pos.numpy(), what="q", **kw)
        _check(ko, base[:, Hq * D:(Hq + Hkv) * D], D, freqs, pos.numpy(), what="k", **kw)
        assert torch.isnan(qo[:, Hq * D:].float()).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved,R", [(False, 64), (False, 36), (True, 64), (True, 20), (False, 32)])
def test_in_place_is_the_same(interleaved, R, dtype):
    T, H, D = 133, 5, 64
    base = _rows(T, H * D, dtype, 3).to(DEV)
    freqs = g.lfm2sc_rotary_freqs(R).to(DEV)
    pos = torch.arange(T, dtype=I32, device=DEV) * 37
    q = base[:, :H * D]
    want = torch.empty(T, H * D, dtype=dtype, device=DEV)
    g.lfm2sc_rotary(q, want, D, freqs, positions=pos, interleaved=interleaved)
    before = base.clone()
    g.lfm2sc_rotary(q, q, D, freqs, positions=pos, interleaved=interleaved)
    assert torch.equal(base[:, :H * D], want) and torch.equal(base[:, H * D:], before[:, H * D:])
    _check(want, before[:, :H * D].cpu(), D, freqs.cpu(), pos.cpu().numpy(), interleaved=interleaved)


@pytest.mark.parametrize("lens", [[1], [5, 0, 0, 130, 1], [0, 0], [3] * 200, [0] * 70 + [9] + [0] * 70])
@pytest.mark.parametrize("starts", [False, True])
def test_packed(lens, starts):
    D, Hq, Hkv, lead, tail = 64, 4, 1, 3, 5
    T = lead + sum(lens) + tail
    base = _rows(T, (Hq + Hkv) * D, BF, len(lens))
    cu = torch.tensor([lead] + lens).cumsum(0).to(I32)
    begin = torch.arange(len(lens), dtype=I32) * 1000 if starts else None
    freqs = g.lfm2sc_rotary_freqs(D, base=1e6)
    x = base.to(DEV)
    qo = torch.full((T, Hq * D), float("nan"), dtype=BF, device=DEV)
    ko = torch.full((T, Hkv * D), float("nan"), dtype=BF, device=DEV)
    g.lfm2sc_rotary(x[:, :Hq * D], qo, D, freqs.to(DEV), positions=None if begin is None else begin.to(DEV), cu_seqlens=cu.to(DEV),
                    k=x[:, Hq * D:(Hq + Hkv) * D], k_out=ko)
    pos, mine = o8.packed_positions(cu.tolist(), T, None if begin is None else begin.tolist())
    for out, cols in ((qo, slice(0, Hq * D)), (ko, slice(Hq * D, (Hq + Hkv) * D))):
        _check(out, base[:, cols], D, freqs, pos, rows=mine)
        assert torch.isnan(out[torch.from_numpy(~mine)].float()).all()


def test_many_rows_and_few_agree_bitwise():
    """One row goes to several waves, many rows to a wave each."""
    D, H, T = 64, 40, 5000
    x = _rows(T, H * D, BF, 1, 0).to(DEV)
    freqs = g.lfm2sc_rotary_freqs(D).to(DEV)
    pos = torch.arange(T, dtype=I32, device=DEV)
    many = g.lfm2sc_rotary(x, torch.empty_like(x), D, freqs, positions=pos)
    for t in (0, 1, 4999):
        assert torch.equal(g.lfm2sc_rotary(x[t:t + 1], torch.empty_like(x[t:t + 1]), D, freqs, positions=pos[t:t + 1]), many[t:t + 1])


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(interleaved):
    """The transposed rotation: <grad, rotate(x)> = <inverse(grad), x>, and against differences of a function of the rows."""
    D, H, T, m = 64, 3, 9, 1.3
    x, w = _rows(T, H * D, F32, 5, 0).to(DEV), _rows(T, H * D, F32, 6, 0).to(DEV)
    freqs = g.lfm2sc_rotary_freqs(48).to(DEV)
    pos = torch.arange(T, dtype=I32, device=DEV) * 11
    kw = dict(positions=pos, interleaved=interleaved, magnitude=m)

    def f(y):                    # sum of w y^3 / 3 over the rotated rows, in 64 bits
        return (w.double() * g.lfm2sc_rotary(y, torch.empty_like(y), D, freqs, **kw).double() ** 3 / 3).sum().item()

    y = g.lfm2sc_rotary(x, torch.empty_like(x), D, freqs, **kw)
    grad = g.lfm2sc_rotary((w * y * y).contiguous(), torch.empty_like(x), D, freqs, inverse=True, **kw)
    left = (w.double() * y.double() ** 2 * y.double()).sum().item()
    right = (grad.double() * x.double()).sum().item()
    terms = (w.double().abs() * y.double().abs() ** 3).sum().item() + (grad.double().abs() * x.double().abs()).sum().item()
    assert abs(left - right) <= 2.0 ** -19 * terms
    gen = torch.Generator().manual_seed(7)
    for _ in range(4):
        d = torch.randn(x.shape, generator=gen).to(DEV)
        h = 2.0 ** -6
        got = (f(x + h * d) - f(x - h * d)) / (2 * h)
        want = (grad.double() * d.double()).sum().item()
        # the cubic's third difference h^2 / 3 sum w dy^3, and fp32 roundings of the rows over h
        dy = g.lfm2sc_rotary(d, torch.empty_like(d), D, freqs, **kw).double()
        bound = h * h / 3 * (w.double().abs() * dy.abs() ** 3).sum().item() + 2.0 ** -20 / h * (
            w.double().abs() * (y.double().abs() + h * dy.abs()) ** 2 * (x.double().abs().max() * 2 * m + 1)).sum().item()
        assert abs(got - want) <= bound, (got, want, bound)


def test_a_nan_stays_in_its_pair():
    D, T = 64, 4
    x = _rows(T, 2 * D, BF, 9, 0)
    x[1, 5], x[2, D + 40] = float("nan"), float("inf")
    freqs = g.lfm2sc_rotary_freqs(32).to(DEV)
    y = g.lfm2sc_rotary(x.to(DEV), torch.empty(T, 2 * D, dtype=BF, device=DEV), D, freqs, positions=torch.arange(T, dtype=I32, device=DEV))
    bad = ~torch.isfinite(y.float()).cpu()
    assert sorted(map(tuple, bad.nonzero().tolist())) == [(1, 5), (1, 21), (2, D + 40)]


def test_rows_past_32_bits():
    D, H, T = 128, 16, (1 << 20) + 5
    x = torch.empty(T, H * D + 8, dtype=BF, device=DEV)      # 4.3 GB
    rows = [0, 1, 524287, 524288, T - 1]
    seed = _rows(len(rows), H * D, BF, 4, 0)
    x[rows, :H * D] = seed.to(DEV)
    freqs = g.lfm2sc_rotary_freqs(D)
    pos = torch.arange(T, dtype=I32, device=DEV)
    g.lfm2sc_rotary(x[:, :H * D], x[:, :H * D], D, freqs.to(DEV), positions=pos)
    _check(x[rows, :H * D].cpu(), seed, D, freqs, np.array(rows))


def test_graph_replays_and_another_stream():
    D, H, T = 64, 8, 33
    x = _rows(T, H * D, BF, 2, 0).to(DEV)
    freqs = g.lfm2sc_rotary_freqs(D).to(DEV)
    pos = torch.arange(T, dtype=I32, device=DEV)
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = g.lfm2sc_rotary(x, torch.empty_like(x), D, freqs, positions=pos)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.lfm2sc_rotary(x, out, D, freqs, positions=pos)
    for shift in (0, 5, 9):
        pos.add_(shift)
        want = g.lfm2sc_rotary(x, torch.empty_like(x), D, freqs, positions=pos)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_at_the_ends_of_their_type(interleaved):
    """Negative positions turn the other way."""
    D, H = 64, 3
    pos = torch.tensor([-2 ** 31, -1, 0, 1, 2 ** 31 - 1], dtype=torch.int32)
    x = torch.randn(5, H * D, generator=torch.Generator().manual_seed(1))
    freqs = g.lfm2sc_rotary_freqs(D)
    y = torch.empty_like(x, device="cuda")
    g.lfm2sc_rotary(x.cuda(), y, D, freqs.cuda(), positions=pos.cuda(), interleaved=interleaved)
    _check(y, x, D, freqs, pos.numpy(), interleaved=interleaved)
