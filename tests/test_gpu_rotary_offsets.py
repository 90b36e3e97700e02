"""Row offsets of lfm2sc_rotary outside [0, total_T] count as clamped, as everywhere in the library (GPU).  Tolerance as in
test_gpu_rotary."""
import pytest
import torch

import gated_short_causal_amd as g
from oracle import cache8 as o8
from test_gpu_rotary import BF, DEV, F32, I32, _check, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu,starts", [([-3, 4, 9], None), ([-3, 4, 9], [7, 100]), ([-(1 << 31), (1 << 31) - 1], [5]), ([-9, -2, 3, 6], None),
                                       ([-1] * 300 + [2, 8], None), ([2, 40, 40], [0, 9])])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_offsets_outside_the_rows(cu, starts, dtype):
    T, D, H = 6, 64, 3
    base = _rows(T, H * D, dtype, 1)
    x, out = base.to(DEV), torch.full((T, H * D), float("nan"), dtype=dtype, device=DEV)
    freqs = g.lfm2sc_rotary_freqs(D)
    g.lfm2sc_rotary(x[:, :H * D], out, D, freqs.to(DEV), cu_seqlens=torch.tensor(cu, dtype=I32, device=DEV),
                    positions=None if starts is None else torch.tensor(starts, dtype=I32, device=DEV))
    inside = [min(max(c, 0), T) for c in cu]
    pos, mine = o8.packed_positions(inside, T, starts)
    _check(out, base[:, :H * D], D, freqs, pos, rows=mine)
    assert torch.isnan(out[torch.from_numpy(~mine)].float()).all()
