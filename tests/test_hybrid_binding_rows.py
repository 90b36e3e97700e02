"""Host checks of what the binding of the hybrid decoder's operators makes of row strides and shapes that the kernels
could not address (no GPU)."""
import pytest
import torch

from gated_short_causal_amd import _lib, binding, hybrid

BF, I32 = torch.bfloat16, torch.int32
SHAPE = 2


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def lib(monkeypatch):
    """CPU tensors pass for GPU tensors."""
    rec = _Recorder()
    monkeypatch.setattr(binding, "_is_gpu", lambda t: True)
    monkeypatch.setattr(binding, "_stream", lambda device: 0)
    monkeypatch.setattr(hybrid._lib, "hybrid_lib", lambda: rec)
    return rec


def _drafts(N=3, L=2, V=11):
    return dict(target_probs=torch.zeros(N * (L + 1), V), draft_tokens=torch.zeros(N, L, dtype=I32), u_accept=torch.zeros(N, L),
                u_sample=torch.zeros(N), accept_len=torch.zeros(N, dtype=I32), next_token=torch.zeros(N, dtype=I32),
                workspace=torch.zeros(4096, dtype=torch.uint8), draft_probs=torch.zeros(N * L, V))


# rows that share memory: one row expanded, and windows 3 elements apart
SHARED = [lambda rows: torch.rand(1, 11).expand(rows, 11), lambda rows: torch.rand(11 + 3 * rows).unfold(0, 11, 3)[:rows]]


@pytest.mark.parametrize("which,rows", [("target_probs", 9), ("draft_probs", 6)])
@pytest.mark.parametrize("make", SHARED)
def test_draft_rows_closer_than_a_row_are_not_spread(lib, which, rows, make):
    """Their stride reaches the library as it is, which refuses one below V."""
    x = make(rows)
    assert x.shape == (rows, 11) and x.stride(0) < 11
    hybrid.lfm2sc_accept_drafts(**{**_drafts(), which: x})
    assert lib.calls[0][1][5 if which == "target_probs" else 7] == x.stride(0)


@pytest.mark.parametrize("ts,ds", [(0, 11), (10, 11), (11, 0), (11, 3)])
def test_the_library_refuses_such_strides(ts, ds):
    P = 0x10000                                      # refused before the first HIP call
    rc = _lib.hybrid_lib().lfm2sc_accept_drafts(1, 11, 3, 2, P, ts, P, ds, P, None, P, P, P, None, P, P, 1 << 20, None)
    assert rc == SHAPE


@pytest.mark.parametrize("make", SHARED)
def test_draft_strides_of_a_single_row_do_not_matter(lib, make):
    """One sequence without drafts has one target row, one with a single draft one draft row: any stride addresses it."""
    a = _drafts(1, 0)
    a.update(target_probs=make(1), draft_probs=None)
    hybrid.lfm2sc_accept_drafts(**a)
    a = _drafts(1, 1)
    a["draft_probs"] = make(1)
    hybrid.lfm2sc_accept_drafts(**a)
    assert lib.calls[0][1][5] == 11 and lib.calls[1][1][7] == 11


def test_true_strides_reach_the_library(lib):
    a = _drafts()
    a.update(target_probs=torch.zeros(9, 16)[:, :11], draft_probs=torch.zeros(6, 13)[:, :11])
    hybrid.lfm2sc_accept_drafts(**a)
    assert lib.calls[0][1][5] == 16 and lib.calls[0][1][7] == 13


def _prompt(T=10, D=64, Hq=4, Hkv=2, **change):
    return {**dict(q=torch.zeros(T, Hq * D, dtype=BF), k=torch.zeros(T, Hkv * D, dtype=BF), v=torch.zeros(T, Hkv * D, dtype=BF),
                   cu_seqlens=torch.tensor([0, T], dtype=I32), D=D, out=torch.zeros(T, Hq * D, dtype=BF), lse=torch.zeros(Hq, T)), **change}


def test_rows_of_another_length_are_refused(lib):
    """lse is read and written as [heads][T], u_accept as [N][L]: a wider matrix holds its rows elsewhere."""
    with pytest.raises(ValueError):
        hybrid.lfm2sc_attn_prefill(**_prompt(lse=torch.zeros(4, 16)))
    a = _prompt(lse=torch.zeros(4, 16))
    a.update(d_out=a["out"], dq=a["q"], dk=a["k"], dv=a["v"], workspace=torch.zeros(1 << 16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        hybrid.lfm2sc_attn_backward(**a)
    with pytest.raises(ValueError):
        hybrid.lfm2sc_accept_drafts(**{**_drafts(), "u_accept": torch.zeros(3, 3)})
    assert lib.calls == []


def test_more_rows_and_flat_buffers_pass(lib):
    hybrid.lfm2sc_attn_prefill(**_prompt(lse=torch.zeros(7, 10)))
    hybrid.lfm2sc_attn_prefill(**_prompt(lse=torch.zeros(64)))
    hybrid.lfm2sc_accept_drafts(**{**_drafts(), "u_accept": torch.zeros(8)})
    hybrid.lfm2sc_accept_drafts(**{**_drafts(), "u_accept": torch.zeros(4, 2)})
    assert len(lib.calls) == 4
