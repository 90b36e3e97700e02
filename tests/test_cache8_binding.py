"""Host checks of the Python binding of the rotary positions and the 8-bit cache (no GPU): what reaches the library, and
refusals before any library call.  The library is a recorder and CPU tensors pass for GPU tensors."""
import pytest
import torch

from gated_short_causal_amd import binding, hybrid
from test_hybrid_binding import _Recorder

BF, I32, F32, E4M3 = torch.bfloat16, torch.int32, torch.float32, torch.float8_e4m3fn


@pytest.fixture
def lib(monkeypatch):
    rec = _Recorder()
    monkeypatch.setattr(hybrid._lib, "hybrid_lib", lambda: rec)
    monkeypatch.setattr(binding, "_is_gpu", lambda t: True)
    monkeypatch.setattr(binding, "_stream", lambda device: 0)
    return rec


def _rot():
    x = torch.zeros(10, 6 * 64 + 8, dtype=BF)
    return dict(q=x[:, :256], q_out=torch.zeros(10, 256, dtype=BF), D=64, freqs=torch.zeros(16), positions=torch.zeros(10, dtype=I32),
                k=x[:, 256:384], k_out=torch.zeros(10, 128, dtype=BF))


def test_rotary_marshals(lib):
    a = _rot()
    hybrid.lfm2sc_rotary(**a, inverse=True, magnitude=1.5)
    hybrid.lfm2sc_rotary(**{**a, "k": None, "k_out": None, "positions": None, "cu_seqlens": torch.zeros(4, dtype=I32)}, interleaved=True)
    (n0, x), (n1, y) = lib.calls
    assert n0 == n1 == "lfm2sc_rotary"
    assert x[:5] == (0, 64, 32, 0, 1) and x[6] == 392 and x[8] == 256 and x[9] == 4 and x[11] == 392 and x[13] == 128 and x[14] == 2
    assert x[15] == 10 and x[16] == a["positions"].data_ptr() and x[17] is None and x[18] == 0 and x[20] == 1.5
    assert y[:5] == (0, 64, 32, 1, 0) and y[10:15] == (None, 0, None, 0, 0) and y[16] is None and y[18] == 3


@pytest.mark.parametrize("change,err", [
    (dict(q_out=torch.zeros(9, 256, dtype=BF)), ValueError), (dict(q_out=torch.zeros(10, 200, dtype=BF)), ValueError),
    (dict(q_out=torch.zeros(10, 512, dtype=BF)), ValueError), (dict(q_out=torch.zeros(10, 256)), TypeError),
    (dict(k_out=None), ValueError), (dict(k=None), ValueError), (dict(k=torch.zeros(10, 128)), TypeError), (dict(positions=None), ValueError),
    (dict(positions=torch.zeros(9, dtype=I32)), ValueError), (dict(positions=torch.zeros(10, dtype=torch.int64)), TypeError),
    (dict(freqs=torch.zeros(16).double()), TypeError), (dict(freqs=torch.zeros(32)[::2]), ValueError), (dict(freqs=torch.zeros(0)), ValueError),
    (dict(cu_seqlens=torch.zeros(12, dtype=I32)), ValueError), (dict(cu_seqlens=torch.zeros(3, dtype=I32)), ValueError), (dict(cu_seqlens=torch.zeros(2, 2, dtype=I32)), ValueError), (dict(D=0), ValueError),
    (dict(q=torch.zeros(10, 256, dtype=torch.float16)), TypeError), (dict(q=torch.zeros(10, 512, dtype=BF)[:, ::2]), ValueError),
])
def test_rotary_refuses(lib, change, err):
    with pytest.raises(err):
        hybrid.lfm2sc_rotary(**{**_rot(), **change})
    assert lib.calls == []


def test_freqs_names(lib):
    with pytest.raises(ValueError):
        hybrid.lfm2sc_rotary_freqs(64, scaling="other")
    assert lib.calls == []
    assert hybrid.lfm2sc_rotary_freqs(64, scaling="parts", factor=8, original_len=8192).shape == (32,)
    assert lib.calls[0][1][:7] == (64, 10000.0, 3, 8, 8192, 1.0, 4.0)


def _cache(P=5, H=2, S=32, D=64, B=16, dtype=E4M3):
    return dict(k_pages=torch.zeros(P, H, S, D, dtype=torch.int8).view(dtype), v_pages=torch.zeros(P, H, S // 16, D, 16, dtype=torch.int8).view(dtype),
                k_scales=torch.zeros(P, H, S // B), v_scales=torch.zeros(P, H, S // B))


def _write():
    kv = torch.zeros(6, 264, dtype=BF)
    return dict(k=kv[:, :128], v=kv[:, 128:256], **_cache(), page_table=torch.zeros(3, 2, dtype=I32), seq_len=torch.zeros(3, dtype=I32))


def _read():
    w = _write()
    w["k_out"], w["v_out"] = w.pop("k"), w.pop("v")
    return w


def _attend():
    return dict(q=torch.zeros(6, 512, dtype=BF), **_cache(), prefix_pages=torch.zeros(4, dtype=I32), prefix_len=100, page_table=torch.zeros(3, 2, dtype=I32),
                suffix_len=torch.zeros(3, dtype=I32), L=2, out=torch.zeros(6, 512, dtype=BF), workspace=torch.zeros(64, dtype=torch.uint8))


CALLS = {"write": (hybrid.lfm2sc_cache8_write, _write), "read": (hybrid.lfm2sc_cache8_read, _read), "attend": (hybrid.lfm2sc_attn_cached8, _attend)}


def test_cache_marshals(lib):
    w = _write()
    hybrid.lfm2sc_cache8_write(**w)
    hybrid.lfm2sc_cache8_write(**{**w, **_cache(dtype=torch.int8)}, cu_seqlens=torch.zeros(4, dtype=I32))
    hybrid.lfm2sc_cache8_read(**_read())
    hybrid.lfm2sc_attn_cached8(**_attend())
    hybrid.lfm2sc_attn_cached8(**_attend(), max_suffix_len=40, scale=0.5)
    (_, a), (_, b), (_, c), (_, d), (_, e) = lib.calls
    assert a[:4] == (0, 0, 64, 2) and a[5] == a[7] == 264 and a[8] == 6 and a[9] is None and a[10] == 3
    assert a[11] == w["k_pages"].data_ptr() and a[13] == 4096 and a[16] == 4 and a[17:20] == (5, 32, 16) and a[21] == 2
    assert b[1] == 1 and b[9] is not None
    assert c[:4] == (0, 0, 64, 2) and c[6] == 4096 and c[9] == 4 and c[10:13] == (5, 32, 16) and c[17] == c[19] == 264 and c[20] == 6 and c[22] == 3
    assert d[:5] == (0, 0, 64, 8, 2) and d[6:9] == (512, 3, 2) and d[11] == 4096 and d[15:18] == (5, 32, 16) and d[19] == 100 and d[21] == 2
    assert d[23] == 64 and d[24] == 0.125 and d[28] == 64
    assert e[23] == 40 and e[24] == 0.5


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("change,err", [
    (dict(k_pages=torch.zeros(5, 2, 32, 64, dtype=torch.uint8)), TypeError), (dict(k_pages=torch.zeros(5, 2, 32, 64)), TypeError),
    (dict(k_pages=torch.zeros(2, 32, 64, dtype=torch.int8)), ValueError), (dict(k_pages=torch.zeros(0, 2, 32, 64, dtype=torch.int8)), ValueError),
    (dict(v_pages=torch.zeros(5, 2, 32, 64, dtype=torch.int8)), ValueError), (dict(v_pages=torch.zeros(5, 2, 2, 64, 16, dtype=torch.int8)), TypeError),
    (dict(v_pages=torch.zeros(4, 2, 2, 64, 16, dtype=torch.int8).view(E4M3)), ValueError),
    (dict(k_scales=torch.zeros(5, 2, 3)), ValueError), (dict(k_scales=torch.zeros(5, 2)), ValueError), (dict(v_scales=torch.zeros(5, 1, 2)), ValueError),
    (dict(k_scales=torch.zeros(5, 2, 2).double()), TypeError), (dict(v_scales=torch.zeros(5, 2, 2, dtype=BF)), TypeError),
    (dict(k_scales=torch.zeros(5, 2, 4)[:, :, ::2]), ValueError), (dict(k_scales=torch.zeros(5, 3, 2)[:, :2]), ValueError),
    (dict(k_pages=torch.zeros(5, 2, 64, 64, dtype=torch.int8).view(E4M3)[:, :, ::2]), ValueError),
    (dict(page_table=torch.zeros(6, dtype=I32)), ValueError), (dict(page_table=torch.zeros(3, 2, dtype=torch.int64)), TypeError),
    (dict(page_table=torch.zeros(3, 4, dtype=I32)[:, ::2]), ValueError),
])
def test_cache_refuses(lib, call, change, err):
    fn, make = CALLS[call]
    with pytest.raises(err):
        fn(**{**make(), **change})
    assert lib.calls == []


@pytest.mark.parametrize("call,change,err", [
    ("write", dict(k=torch.zeros(6, 120, dtype=BF)), ValueError), ("write", dict(v=torch.zeros(5, 128, dtype=BF)), ValueError),
    ("write", dict(v=torch.zeros(6, 128)), TypeError), ("write", dict(k=torch.zeros(6, 128, dtype=torch.float16)), TypeError),
    ("write", dict(seq_len=torch.zeros(2, dtype=I32)), ValueError), ("write", dict(seq_len=None), ValueError),
    ("write", dict(cu_seqlens=torch.zeros(3, dtype=I32)), ValueError), ("write", dict(cu_seqlens=torch.zeros(4)), TypeError),
    ("read", dict(k_out=torch.zeros(6, 120, dtype=BF)), ValueError), ("read", dict(v_out=torch.zeros(6, 128)), TypeError),
    ("read", dict(seq_len=torch.zeros(3)), TypeError),
    ("attend", dict(q=torch.zeros(5, 512, dtype=BF)), ValueError), ("attend", dict(out=torch.zeros(6, 500, dtype=BF)), ValueError),
    ("attend", dict(prefix_pages=torch.zeros(3, dtype=I32)), ValueError), ("attend", dict(prefix_pages=None), ValueError),
    ("attend", dict(suffix_len=torch.zeros(2, dtype=I32)), ValueError), ("attend", dict(workspace=torch.zeros(64)[::2]), ValueError),
])
def test_calls_refuse(lib, call, change, err):
    fn, make = CALLS[call]
    with pytest.raises(err):
        fn(**{**make(), **change})
    assert lib.calls == []


def test_k_and_v_in_one_pool(lib):
    """Pages of k and v side by side, scales with room: the strides of a page reach the library."""
    pool, scales = torch.zeros(5, 2, 4096, dtype=torch.int8), torch.zeros(5, 2, 8)
    c = dict(k_pages=pool[:, 0].view(5, 2, 32, 64), v_pages=pool[:, 1].view(5, 2, 2, 64, 16), k_scales=scales[:, 0, :4].view(5, 2, 2),
             v_scales=scales[:, 1, :4].view(5, 2, 2))
    hybrid.lfm2sc_cache8_write(**{**_write(), **c})
    assert lib.calls[0][1][13] == 8192 and lib.calls[0][1][16] == 16
    with pytest.raises(ValueError):
        hybrid.lfm2sc_cache8_write(**{**_write(), **c, "v_pages": torch.zeros(5, 2, 2, 64, 16, dtype=torch.int8)})


def test_cpu_tensors_are_refused():
    for call, (fn, make) in CALLS.items():
        with pytest.raises(ValueError):
            fn(**make())
    with pytest.raises(ValueError):
        hybrid.lfm2sc_rotary(**_rot())
