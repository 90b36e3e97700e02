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


def test_workspace_queries_at_extreme_sizes(L):
    """Sizes are computed in 64 bits: never negative or wrapped (the caller would allocate too little)."""
    ends = (-(1 << 31), -1, 0, 1, 31, 1 << 14, (1 << 24) - 1, (1 << 30) - 1, 1 << 30, (1 << 31) - 1)
    for H, Hkv in ((1, 1), (32, 8), (1 << 14, 1), (1 << 14, 1 << 14)):
        for n in ends:
            for T in ends + (1 << 40,):
                got = L.lfm2sc_attn_backward_workspace_bytes(0, 128, H, Hkv, T, n)
                valid = n > 0 and 0 < T < 1 << 30
                assert (got >= 8 * H * T) if valid else got == 0, (H, Hkv, T, n)
            for block in ends:
                for prefix in ends:
                    for pages, page in ((0, 16), (1, 1 << 29), (1 << 25, 16), (1 << 29, 4), (-1, 16), (4, 12)):
                        got = L.lfm2sc_attn_cached_workspace_bytes(0, 128, H, Hkv, n, block, prefix, pages, page)
                        valid = (n > 0 and block > 0 and n * block * H < 1 << 28 and 0 <= prefix < 1 << 30 and pages >= 0
                                 and page & (page - 1) == 0 and pages * page < 1 << 30)
                        assert valid or got == 0, (H, n, block, prefix, pages, page)
                        # the split form keeps at least one partial row of D and a pair per row of each part
                        assert got == 0 or got >= n * block * H * (128 * 4 + 8), (H, n, block, prefix, pages, page)


@pytest.mark.parametrize("N,block,H", [(1 << 20, 1 << 30, 1 << 14), ((1 << 31) - 1, (1 << 31) - 1, 32), (1 << 30, 1 << 30, 16)])
def test_cached_sizes_whose_product_passes_64_bits(L, N, block, H):
    assert L.lfm2sc_attn_cached_workspace_bytes(0, 64, H, 1, N, block, 500, 4, 16) == 0
    assert L.lfm2sc_attn_cached(0, 64, H, 1, P, H * 64, N, block, P, P, 64, 1000, 16, P, 500, P, 4, P, 0.125, P, H * 64, P, HUGE,
                                None) == SHAPE


def test_draft_workspace_query_at_extreme_sizes(L):
    ends = (-(1 << 31), -1, 0, 1, 4096, 4097, (1 << 30) - 1, 1 << 30, (1 << 31) - 4096, (1 << 31) - 1)
    for n in ends:
        for V in ends:
            got = L.lfm2sc_accept_drafts_workspace_bytes(n, 4, V)
            if n > 0 and 0 < V < 1 << 30:
                assert n * 2 * -(-V // 4096) * 8 <= got < n * 2 * -(-V // 4096) * 8 + 256, (n, V)
            else:
                assert got == 0, (n, V)
