"""Host checks of the Python binding of the hybrid decoder's operators (no GPU): refusals before any library call, and
the sizes and strides that reach it.  The library is a recorder and CPU tensors pass for GPU tensors."""
import pytest
import torch

from gated_short_causal_amd import binding, hybrid

BF, I32, F32 = torch.bfloat16, torch.int32, torch.float32


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
    rec = _Recorder()
    monkeypatch.setattr(hybrid._lib, "hybrid_lib", lambda: rec)
    monkeypatch.setattr(binding, "_is_gpu", lambda t: True)
    monkeypatch.setattr(binding, "_stream", lambda device: 0)
    return rec


def _prompt(T=10, D=64, Hq=4, Hkv=2):
    qkv = torch.zeros(T, (Hq + 2 * Hkv) * D, dtype=BF)
    return dict(q=qkv[:, :Hq * D], k=qkv[:, Hq * D:(Hq + Hkv) * D], v=qkv[:, (Hq + Hkv) * D:], cu_seqlens=torch.tensor([0, 4, T], dtype=I32),
                D=D, out=torch.zeros(T, Hq * D, dtype=BF), lse=torch.zeros(Hq, T))


def test_prefill_marshals(lib):
    a = _prompt()
    hybrid.lfm2sc_attn_prefill(**a)
    (name, args), = lib.calls
    assert name == "lfm2sc_attn_prefill"
    assert args[:4] == (0, 64, 4, 2) and args[5] == args[7] == args[9] == 512 and args[10] == 10 and args[12] == 2
    assert args[13] == 0.125 and args[15] == 256 and args[16] == a["lse"].data_ptr()
    hybrid.lfm2sc_attn_prefill(**{**a, "lse": None, "scale": 2})
    assert lib.calls[1][1][13] == 2.0 and lib.calls[1][1][16] is None


@pytest.mark.parametrize("change,err", [
    (dict(k=torch.zeros(9, 128, dtype=BF)), ValueError), (dict(v=torch.zeros(10, 64, dtype=BF)), ValueError),
    (dict(k=torch.zeros(10, 128)), TypeError), (dict(out=torch.zeros(10, 200, dtype=BF)), ValueError),
    (dict(out=torch.zeros(9, 256, dtype=BF)), ValueError), (dict(out=torch.zeros(10, 512, dtype=BF)), ValueError),
    (dict(cu_seqlens=torch.zeros(3, dtype=torch.int64)), TypeError), (dict(cu_seqlens=None), ValueError),
    (dict(lse=torch.zeros(3, 10)), ValueError), (dict(lse=torch.zeros(4, 10, dtype=BF)), TypeError),
    (dict(q=torch.zeros(10, 512, dtype=BF)[:, ::2]), ValueError), (dict(D=0), ValueError),
])
def test_prefill_refuses(lib, change, err):
    with pytest.raises(err):
        hybrid.lfm2sc_attn_prefill(**{**_prompt(), **change})
    assert lib.calls == []


def _bwd():
    a = _prompt()
    a.update(d_out=torch.zeros_like(a["out"]), dq=torch.zeros(10, 256, dtype=BF), dk=torch.zeros(10, 128, dtype=BF),
             dv=torch.zeros(10, 136, dtype=BF), workspace=torch.zeros(100, dtype=torch.uint8))
    return a


def test_backward_marshals(lib):
    a = _bwd()
    hybrid.lfm2sc_attn_backward(**a)
    (_, args), = lib.calls
    assert args[18] == 256 and args[20] == 256 and args[22] == 128 and args[24] == 136 and args[26] == 100


@pytest.mark.parametrize("change,err", [
    (dict(lse=None), ValueError), (dict(d_out=torch.zeros(9, 256, dtype=BF)), ValueError), (dict(dq=torch.zeros(10, 256)), TypeError),
    (dict(dk=torch.zeros(10, 64, dtype=BF)), ValueError), (dict(dv=torch.zeros(5, 128, dtype=BF)), ValueError),
    (dict(workspace=torch.zeros(100, dtype=torch.uint8)[::2]), ValueError),
])
def test_backward_refuses(lib, change, err):
    with pytest.raises(err):
        hybrid.lfm2sc_attn_backward(**{**_bwd(), **change})
    assert lib.calls == []


def _cached():
    pool = torch.zeros(10, 16, 2, 2, 64, dtype=BF)     # k and v of a token next to each other
    return dict(q=torch.zeros(6, 256, dtype=BF), k_pages=pool[:, :, 0], v_pages=pool[:, :, 1], prefix_pages=torch.zeros(2, dtype=I32),
                prefix_len=20, page_table=torch.zeros(3, 4, dtype=I32), suffix_len=torch.zeros(3, dtype=I32), L=2,
                out=torch.zeros(6, 256, dtype=BF), workspace=torch.zeros(64, dtype=torch.uint8))


def test_cached_marshals(lib):
    hybrid.lfm2sc_attn_cached(**_cached())
    (_, args), = lib.calls
    assert args[:4] == (0, 64, 4, 2) and args[5:8] == (256, 3, 2) and args[10:13] == (256, 10, 16) and args[14] == 20
    assert args[16] == 4 and args[20] == 256 and args[22] == 64
    hybrid.lfm2sc_attn_cached(**{**_cached(), "prefix_pages": None, "prefix_len": 0})
    assert lib.calls[1][1][13] is None


@pytest.mark.parametrize("change,err", [
    (dict(k_pages=torch.zeros(10, 16, 2, 128, dtype=BF)), ValueError), (dict(v_pages=torch.zeros(9, 16, 2, 64, dtype=BF)), ValueError),
    (dict(k_pages=torch.zeros(160, 2, 64, dtype=BF)), ValueError), (dict(q=torch.zeros(5, 256, dtype=BF)), ValueError),
    (dict(out=torch.zeros(6, 100, dtype=BF)), ValueError), (dict(prefix_pages=None), ValueError),
    (dict(prefix_pages=torch.zeros(1, dtype=I32)), ValueError), (dict(page_table=torch.zeros(3, 4)), TypeError),
    (dict(page_table=torch.zeros(12, dtype=I32)), ValueError), (dict(suffix_len=torch.zeros(2, dtype=I32)), ValueError),
    (dict(page_table=torch.zeros(3, 8, dtype=I32)[:, ::2]), ValueError), (dict(q=torch.zeros(6, 256)), TypeError),
])
def test_cached_refuses(lib, change, err):
    with pytest.raises(err):
        hybrid.lfm2sc_attn_cached(**{**_cached(), **change})
    assert lib.calls == []


@pytest.mark.parametrize("pool", [torch.zeros(10, 16, 4, 64, dtype=BF)[:, :, ::2], torch.zeros(20, 16, 2, 64, dtype=BF)[::2],
                                  torch.zeros(10, 2, 16, 64, dtype=BF).transpose(1, 2)])
def test_cached_refuses_other_page_layouts(lib, pool):
    with pytest.raises(ValueError):
        hybrid.lfm2sc_attn_cached(**{**_cached(), "k_pages": pool, "v_pages": pool})
    assert lib.calls == []


def _drafts():
    return dict(target_probs=torch.zeros(9, 11), draft_tokens=torch.zeros(3, 2, dtype=I32), u_accept=torch.zeros(3, 2),
                u_sample=torch.zeros(3), accept_len=torch.zeros(3, dtype=I32), next_token=torch.zeros(3, dtype=I32),
                workspace=torch.zeros(64, dtype=torch.uint8), draft_probs=torch.zeros(6, 16)[:, :11], keep_len=torch.zeros(3, dtype=I32))


def test_drafts_marshal(lib):
    hybrid.lfm2sc_accept_drafts(**_drafts())
    (_, args), = lib.calls
    assert args[:4] == (1, 11, 3, 2) and args[5] == 11 and args[7] == 16 and args[9] is None and args[16] == 64


@pytest.mark.parametrize("change,err", [
    (dict(target_probs=torch.zeros(8, 11)), ValueError), (dict(draft_probs=torch.zeros(6, 10)), ValueError),
    (dict(draft_probs=torch.zeros(6, 11, dtype=BF)), TypeError), (dict(draft_tokens=torch.zeros(6, dtype=I32)), ValueError),
    (dict(draft_tokens=torch.zeros(3, 2)), TypeError), (dict(u_accept=torch.zeros(5)), ValueError),
    (dict(u_sample=torch.zeros(3, dtype=torch.float64)), TypeError), (dict(accept_len=torch.zeros(2, dtype=I32)), ValueError),
    (dict(next_token=torch.zeros(3)), TypeError), (dict(keep_len=torch.zeros(3)), TypeError),
    (dict(num_drafts=torch.zeros(1, dtype=I32)), ValueError), (dict(target_probs=torch.zeros(9, 11, dtype=torch.float16)), TypeError),
])
def test_drafts_refuse(lib, change, err):
    with pytest.raises(err):
        hybrid.lfm2sc_accept_drafts(**{**_drafts(), **change})
    assert lib.calls == []


def test_cpu_tensors_are_refused():
    with pytest.raises(ValueError):
        hybrid.lfm2sc_attn_prefill(**_prompt())
    with pytest.raises(ValueError):
        hybrid.lfm2sc_attn_cached(**_cached())
    with pytest.raises(ValueError):
        hybrid.lfm2sc_accept_drafts(**_drafts())
