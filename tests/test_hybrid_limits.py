"""A launch holds fewer than 2^32 work-items a dimension.  Calls that need more are refused before the first HIP call (CPU;
the pointers are fake and only refused calls are made)."""
import pytest

from gated_short_causal_amd import _lib

SHAPE, P, HUGE = 2, 0x10000, 1 << 60


@pytest.fixture(scope="module")
def L():
    return _lib.hybrid_lib()


# half a million sequences of one token, 32 heads: 2^24 workgroups of 256; and tokens whose delta alone has 2^32
@pytest.mark.parametrize("T,N,H,Hkv", [(1 << 19, 1 << 19, 32, 8), (1 << 19, 1 << 19, 32, 32)])
@pytest.mark.parametrize("D", [64, 128])
def test_prompts(L, T, N, H, Hkv, D):
    q = (P, H * D, P, Hkv * D, P, Hkv * D, T, P, N, 0.125, P, H * D)
    assert L.lfm2sc_attn_prefill(0, D, H, Hkv, *q, P, None) == SHAPE
    assert "work-items" in L.lfm2sc_last_error().decode()
    assert L.lfm2sc_attn_backward(0, D, H, Hkv, *q, P, P, H * D, P, H * D, P, Hkv * D, P, Hkv * D, P, HUGE, None) == SHAPE


def test_delta_of_the_backward(L):
    T = 1 << 29
    q = (P, 64, P, 64, P, 64, T, P, 1, 0.125, P, 64)
    assert L.lfm2sc_attn_backward(0, 64, 1, 1, *q, P, P, 64, P, 64, P, 64, P, 64, P, HUGE, None) == SHAPE


# 2^26 rows to join, a workgroup of 4 rows each; with and without a prefix, split and (N * heads small) direct
@pytest.mark.parametrize("N,block,H,Hkv,prefix", [(1 << 21, 1, 32, 8, 500), (1, 1 << 21, 32, 1, 500), (1 << 25, 1, 4, 1, 0)])
def test_cached(L, N, block, H, Hkv, prefix):
    assert L.lfm2sc_attn_cached(0, 64, H, Hkv, P, H * 64, N, block, P, P, Hkv * 64, 1000, 16, P, prefix, P, 4, P, 0.125, P,
                                H * 64, P, HUGE, None) == SHAPE


def test_drafts(L):
    N = 1 << 22                                     # a workgroup of 1024 each
    assert L.lfm2sc_accept_drafts(1, 16, N, 1, P, 16, P, 16, P, P, P, P, P, P, P, P, HUGE, None) == SHAPE
