"""Python binding of include/lfm2sc_hybrid.h: attention over packed prompts and over a paged cache (bf16, or 8-bit codes
that are quantised as they are written), rotary positions, and draft verification, in the manner of ``binding``: the C entry points' names, torch tensors in, caller-owned outputs
written in place on the current stream, and checks of everything visible in the tensors before any library call.

Tensor conventions (see the header for the full contract):
  q, out, gradients  [rows, >= heads*D]  bf16, unit column stride; the number of heads is the width over D
  k, v               [rows, kv_heads*D]
  k_pages, v_pages   [pages, page_size, kv_heads, D] bf16, the last two dense, pages evenly spaced
  8-bit pages        k [pages, kv_heads, page_size, D], v [pages, kv_heads, page_size/16, D, 16], float8_e4m3fn or int8, dense
                     within a page; scales [pages, kv_heads, page_size/scale_tokens] fp32
  target_probs       [N*(L+1), V], draft_probs [N*L, V], bf16 or fp32
"""
import torch

from . import _lib, binding
from .binding import _check, _dtype_code, _ptr

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32

# The checks run in every call, and a small call's time is mostly the host's: each looks at a tensor once, and the
# wording of a refusal is only worked out when one is due.


def _gpu(ref, name):
    """The index of ref's GPU."""
    if not binding._is_gpu(ref):
        raise ValueError(f"{name} must be a GPU tensor, got device {ref.device}")
    return ref.get_device()


def _refuse(t, name, dev, dtype, what):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be {what}, got {t!r:.100}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the first tensor's GPU, got {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be {what}, got shape {tuple(t.shape)} strides {t.stride()}")


def _mat(t, name, dev, dtype, rows, cols):
    """Row stride of a matrix of at least rows x cols with unit column stride.  Where the call addresses one row at most,
    a stride below its width means nothing and the width stands in; else it goes to the library, which refuses it."""
    if t.dtype is dtype and t.get_device() == dev:
        shape = t.shape
        if len(shape) != 2:
            _refuse(t, name, dev, dtype, "a matrix")
        r, c = shape
        s, unit = t.stride()
        if r >= rows and c >= cols and (unit == 1 or c <= 1):
            return s if s >= cols or rows > 1 else cols
    _refuse(t, name, dev, dtype, f"a matrix of at least [{rows}, {cols}] with unit column stride")


def _vec(t, name, dev, dtype, numel, width=None):
    """Address of a contiguous tensor of at least numel entries, a matrix in rows of `width`; None for None."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == dev and t.numel() >= numel and t.is_contiguous():
        if width is None or t.dim() != 2 or t.shape[1] == width:
            return t.data_ptr()
        _refuse(t, name, dev, dtype, f"in rows of {width} entries")
    _refuse(t, name, dev, dtype, f"contiguous with at least {numel} entries")


def _needed(t, name, dev, dtype, numel, width=None):
    if t is None:
        raise ValueError(f"{name} is required")
    return _vec(t, name, dev, dtype, numel, width)


def _heads(width, D, name):
    if D <= 0 or width % D != 0:
        raise ValueError(f"{name} is {width} columns wide, not a multiple of the head dimension {D}")
    return width // D


def _workspace(t, dev):
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        _refuse(t, "workspace", dev, t.dtype, "contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def _prompt(q, k, v, cu_seqlens, D, out, lse, scale):
    """The arguments that the forward and the backward share, up to out's stride."""
    dev = _gpu(q, "q")
    dtype = q.dtype
    T = q.shape[0]
    Hq, Hkv = _heads(out.shape[-1], D, "out"), _heads(k.shape[-1], D, "k")
    if cu_seqlens is None or cu_seqlens.dim() != 1:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor of N+1 row offsets")
    cu = _vec(cu_seqlens, "cu_seqlens", dev, _I32, 1)
    return dev, (_dtype_code(q), D, Hq, Hkv, q.data_ptr(), _mat(q, "q", dev, dtype, T, Hq * D),
                 k.data_ptr(), _mat(k, "k", dev, dtype, T, Hkv * D), v.data_ptr(), _mat(v, "v", dev, dtype, T, Hkv * D),
                 T, cu, cu_seqlens.numel() - 1, D ** -0.5 if scale is None else scale,
                 out.data_ptr(), _mat(out, "out", dev, dtype, T, Hq * D)), _vec(lse, "lse", dev, _F32, Hq * T, T)


def lfm2sc_attn_prefill(q, k, v, cu_seqlens, D, out, lse=None, scale=None):
    """Causal attention with grouped heads over packed prompts; writes out, and lse ([heads, T] fp32) when given.
    scale defaults to D ** -0.5."""
    _, args, lse = _prompt(q, k, v, cu_seqlens, D, out, lse, scale)
    rc = _lib.hybrid_lib().lfm2sc_attn_prefill(*args, lse, binding._stream(q.device))
    if rc:
        _check(rc)
    return out


def lfm2sc_attn_backward_workspace_bytes(dtype, D, num_heads, num_kv_heads, total_T, num_seqs) -> int:
    code = binding._DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_lib.hybrid_lib().lfm2sc_attn_backward_workspace_bytes(code, D, num_heads, num_kv_heads, total_T, num_seqs))


def lfm2sc_attn_backward(q, k, v, cu_seqlens, D, out, lse, d_out, dq, dk, dv, workspace, scale=None):
    """Backward of lfm2sc_attn_prefill: writes dq, dk and dv (summed over each group's heads)."""
    dev, args, lse = _prompt(q, k, v, cu_seqlens, D, out, lse, scale)
    if lse is None:
        raise ValueError("lse of the forward is required")
    dtype, T, wq, wk = q.dtype, args[10], args[2] * D, args[3] * D
    rc = _lib.hybrid_lib().lfm2sc_attn_backward(
        *args, lse, d_out.data_ptr(), _mat(d_out, "d_out", dev, dtype, T, wq), dq.data_ptr(), _mat(dq, "dq", dev, dtype, T, wq),
        dk.data_ptr(), _mat(dk, "dk", dev, dtype, T, wk), dv.data_ptr(), _mat(dv, "dv", dev, dtype, T, wk),
        *_workspace(workspace, dev), binding._stream(q.device))
    if rc:
        _check(rc)
    return dq, dk, dv


def lfm2sc_attn_cached_workspace_bytes(dtype, D, num_heads, num_kv_heads, num_seqs, L, prefix_len, max_pages,
                                       page_size) -> int:
    code = binding._DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_lib.hybrid_lib().lfm2sc_attn_cached_workspace_bytes(code, D, num_heads, num_kv_heads, num_seqs, L,
                                                                    prefix_len, max_pages, page_size))


def _pages(t, name):
    """(pages, page_size, kv_heads, D, token stride) of a page pool."""
    if t.dim() != 4 or t.numel() == 0:
        raise ValueError(f"{name} must be a [pages, page_size, kv_heads, D] tensor, got shape {tuple(t.shape)}")
    P, S, H, D = t.shape
    sp, st, sh, sd = t.stride()
    if S == 1:
        st = sp if P > 1 else H * D
    if sd != 1 or (H > 1 and sh != D):
        raise ValueError(f"{name}: a token's heads must be dense, got strides {t.stride()}")
    if P > 1 and sp != S * st:
        raise ValueError(f"{name}: pages must be {S} token strides apart, got strides {t.stride()}")
    return P, S, H, D, st


def lfm2sc_attn_cached(q, k_pages, v_pages, prefix_pages, prefix_len, page_table, suffix_len, L, out, workspace,
                       scale=None):
    """Attention of L new tokens per sequence (q [N*L, heads*D], the rows of a verify block; L = 1: decode) over a paged
    cache: the prefix_len keys of prefix_pages, shared by the batch, then each sequence's own suffix_len keys (the new ones
    included) in its page_table row [N, max_pages]."""
    dev = _gpu(q, "q")
    dtype = q.dtype
    P, S, Hkv, D, stride = _pages(k_pages, "k_pages")
    if k_pages.shape != v_pages.shape or k_pages.stride() != v_pages.stride():
        raise ValueError("k_pages and v_pages must have the same shape and strides")
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if t.dtype is not dtype or t.get_device() != dev:
            _refuse(t, name, dev, dtype, "a page pool")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [N, max_pages]")
    N, most = page_table.shape
    table = _vec(page_table, "page_table", dev, _I32, 0)
    lens = _needed(suffix_len, "suffix_len", dev, _I32, N)
    prefix = _needed(prefix_pages, "prefix_pages", dev, _I32, -(-prefix_len // S)) if prefix_len > 0 else None
    Hq = _heads(out.shape[-1], D, "out")
    rc = _lib.hybrid_lib().lfm2sc_attn_cached(
        _dtype_code(q), D, Hq, Hkv, q.data_ptr(), _mat(q, "q", dev, dtype, N * L, Hq * D), N, L, k_pages.data_ptr(),
        v_pages.data_ptr(), stride, P, S, prefix, prefix_len, table, most, lens, D ** -0.5 if scale is None else scale,
        out.data_ptr(), _mat(out, "out", dev, dtype, N * L, Hq * D), *_workspace(workspace, dev), binding._stream(q.device))
    if rc:
        _check(rc)
    return out


def lfm2sc_accept_drafts_workspace_bytes(num_seqs, L, V) -> int:
    return int(_lib.hybrid_lib().lfm2sc_accept_drafts_workspace_bytes(num_seqs, L, V))


def lfm2sc_accept_drafts(target_probs, draft_tokens, u_accept, u_sample, accept_len, next_token, workspace,
                         draft_probs=None, num_drafts=None, keep_len=None):
    """Speculative verification: accept_len [N] drafts of draft_tokens [N, L] are kept, next_token [N] is drawn from what
    is left; keep_len [N] = accept_len + 1 is the accept length lfm2sc_commit_window takes for a block that starts with
    the last sampled token.  u_accept [N, L], u_sample [N]: uniform fp32 numbers in [0, 1)."""
    dev = _gpu(target_probs, "target_probs")
    dtype = target_probs.dtype
    if draft_tokens.dim() != 2:
        raise ValueError("draft_tokens must be [N, L]")
    N, L = draft_tokens.shape
    V = target_probs.shape[-1]
    ts = _mat(target_probs, "target_probs", dev, dtype, N * (L + 1), V)
    ds = V if draft_probs is None else _mat(draft_probs, "draft_probs", dev, dtype, N * L, V)
    rc = _lib.hybrid_lib().lfm2sc_accept_drafts(
        _dtype_code(target_probs), V, N, L, target_probs.data_ptr(), ts, _ptr(draft_probs), ds,
        _vec(draft_tokens, "draft_tokens", dev, _I32, 0), _vec(num_drafts, "num_drafts", dev, _I32, N),
        _needed(u_accept, "u_accept", dev, _F32, N * L, L), _needed(u_sample, "u_sample", dev, _F32, N),
        _needed(accept_len, "accept_len", dev, _I32, N), _vec(keep_len, "keep_len", dev, _I32, N),
        _needed(next_token, "next_token", dev, _I32, N), *_workspace(workspace, dev), binding._stream(target_probs.device))
    if rc:
        _check(rc)
    return accept_len, next_token


_ROPE = {"plain": 0, "linear": 1, "base": 2, "parts": 3}


def lfm2sc_rotary_freqs(rotary_dim, base=10000.0, scaling="plain", factor=1.0, original_len=0.0, low=1.0, high=4.0):
    """The [rotary_dim / 2] fp32 frequencies (a CPU tensor) that lfm2sc_rotary takes: base^(-2i / rotary_dim), scaled for longer
    contexts by "linear" (over factor), "base" (base grows) or "parts" (pairs that turn fewer than low times over original_len
    tokens are slowed by factor, those above high stay)."""
    if scaling not in _ROPE:
        raise ValueError(f"scaling must be one of {', '.join(_ROPE)}, got {scaling!r:.100}")
    freqs = torch.empty(max(0, rotary_dim // 2), dtype=_F32)
    rc = _lib.hybrid_lib().lfm2sc_rotary_freqs(rotary_dim, base, _ROPE[scaling], factor, original_len, low, high, freqs.data_ptr())
    if rc:
        _check(rc)
    return freqs


def lfm2sc_rotary(q, q_out, D, freqs, positions=None, cu_seqlens=None, k=None, k_out=None, interleaved=False, inverse=False,
                  magnitude=1.0):
    """Rotary positions of the rows of q [T, heads*D] and, when given, k [T, kv_heads*D]: the first 2 * len(freqs) columns of
    every head turn by position * freqs.  positions [T]; or with cu_seqlens [N+1] the position of each sequence's first row [N]
    (None: 0).  q_out may be q and k_out k.  inverse=True: the gradient.  float32 or bfloat16."""
    dev = _gpu(q, "q")
    dtype = q.dtype
    code = _dtype_code(q)
    T = q.shape[0]
    Hq = _heads(q_out.shape[-1], D, "q_out")
    qs, qos = _mat(q, "q", dev, dtype, T, Hq * D), _mat(q_out, "q_out", dev, dtype, T, Hq * D)
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    if k is None:
        Hkv, kp, ks, kop, kos = 0, None, 0, None, 0
    else:
        Hkv = _heads(k_out.shape[-1], D, "k_out")
        kp, ks = k.data_ptr(), _mat(k, "k", dev, dtype, T, Hkv * D)
        kop, kos = k_out.data_ptr(), _mat(k_out, "k_out", dev, dtype, T, Hkv * D)
    if cu_seqlens is None:
        N, cu, pos = 0, None, _needed(positions, "positions", dev, _I32, T)
    else:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be a 1-D int32 tensor of N+1 row offsets")
        N = cu_seqlens.numel() - 1
        cu, pos = _vec(cu_seqlens, "cu_seqlens", dev, _I32, 1), _vec(positions, "positions", dev, _I32, N)
        if pos is not None and positions.numel() != N:
            raise ValueError(f"with cu_seqlens, positions are those of the {N} sequences' first rows, got {positions.numel()}")
    rc = _lib.hybrid_lib().lfm2sc_rotary(
        code, D, 2 * freqs.numel(), int(interleaved), int(inverse), q.data_ptr(), qs, q_out.data_ptr(), qos, Hq, kp, ks, kop, kos,
        Hkv, T, pos, cu, N, _vec(freqs, "freqs", dev, _F32, 1), magnitude, binding._stream(q.device))
    if rc:
        _check(rc)
    return q_out if k is None else (q_out, k_out)


_FORMATS = {torch.float8_e4m3fn: 0, torch.int8: 1}


def _dense(t, name, inner):
    """A pool's page stride; a page is dense (strides `inner`, which mean nothing where a size is 1)."""
    stride = t.stride()
    if stride[1:] != inner and any(n > 1 and a != b for n, a, b in zip(t.shape[1:], stride[1:], inner)):
        raise ValueError(f"{name} must be dense within a page, got shape {tuple(t.shape)} strides {stride}")
    return stride[0]


def _pool8(k_pages, v_pages, k_scales, v_scales, dev):
    """(format, D, kv_heads, (addresses and strides of the pools, pages, page_size, scale_tokens)) of an 8-bit cache."""
    dtype, shape = k_pages.dtype, k_pages.shape
    fmt = _FORMATS.get(dtype)
    if fmt is None:
        raise TypeError(f"k_pages must be torch.float8_e4m3fn or torch.int8, got {dtype}")
    if len(shape) != 4 or 0 in shape:
        raise ValueError(f"k_pages must be a [pages, kv_heads, page_size, D] tensor, got shape {tuple(shape)}")
    P, H, S, D = shape
    if v_pages.shape != (P, H, S // 16, D, 16):
        raise ValueError(f"v_pages must be [pages, kv_heads, page_size / 16, D, 16] = {(P, H, S // 16, D, 16)}, got "
                         f"{tuple(v_pages.shape)}")
    scales = k_scales.shape
    B = scales[2] if len(scales) == 3 else 0
    if B < 1 or S % B != 0 or scales != (P, H, B) or v_scales.shape != scales:
        raise ValueError(f"k_scales and v_scales must be [pages, kv_heads, page_size / scale_tokens] of {P} pages, {H} heads and "
                         f"{S} tokens, got {tuple(scales)} and {tuple(v_scales.shape)}")
    for name, t, want in (("k_pages", k_pages, dtype), ("v_pages", v_pages, dtype), ("k_scales", k_scales, _F32),
                          ("v_scales", v_scales, _F32)):
        if t.dtype is not want or t.get_device() != dev:
            _refuse(t, name, dev, want, "part of the cache")
    page = S * D
    ps, ss = _dense(k_pages, "k_pages", (page, D, 1)), _dense(k_scales, "k_scales", (B, 1))
    pv, sv = _dense(v_pages, "v_pages", (page, 16 * D, 16, 1)), _dense(v_scales, "v_scales", (B, 1))
    if P == 1:
        ps, ss = H * page, H * B
    elif pv != ps or sv != ss:
        raise ValueError("the pages of k and of v, and their scales, must be evenly spaced alike")
    return fmt, D, H, (k_pages.data_ptr(), v_pages.data_ptr(), ps, k_scales.data_ptr(), v_scales.data_ptr(), ss, P, S, S // B)


def _table(page_table, lens, name, dev):
    """(N, (page_table's address, max_pages, the lengths' address))"""
    shape = page_table.shape
    if len(shape) != 2:
        raise ValueError("page_table must be [N, max_pages]")
    return shape[0], (_vec(page_table, "page_table", dev, _I32, 0), shape[1], _needed(lens, name, dev, _I32, shape[0]))


def _rows8(k, v, width, cu_seqlens, N, dev, names):
    dtype, T = k.dtype, k.shape[0]
    if cu_seqlens is not None and (cu_seqlens.dim() != 1 or cu_seqlens.numel() != N + 1):
        raise ValueError(f"cu_seqlens must be a 1-D int32 tensor of {N + 1} row offsets")
    return ((k.data_ptr(), _mat(k, names[0], dev, dtype, T, width), v.data_ptr(), _mat(v, names[1], dev, dtype, T, width), T),
            _vec(cu_seqlens, "cu_seqlens", dev, _I32, 1))


def lfm2sc_cache8_write(k, v, k_pages, v_pages, k_scales, v_scales, page_table, seq_len, cu_seqlens=None):
    """Quantises the rows of k and v [T, kv_heads*D] (bf16 or fp32) into the 8-bit cache, as the newest tokens of the sequences:
    seq_len [N] counts them in.  Rows are packed by cu_seqlens [N+1], or T / N to every sequence.  page_table [N, max_pages]."""
    dev = _gpu(k, "k")
    fmt, D, H, pool = _pool8(k_pages, v_pages, k_scales, v_scales, dev)
    N, where = _table(page_table, seq_len, "seq_len", dev)
    rows, cu = _rows8(k, v, H * D, cu_seqlens, N, dev, ("k", "v"))
    rc = _lib.hybrid_lib().lfm2sc_cache8_write(_dtype_code(k), fmt, D, H, *rows, cu, N, *pool, *where, binding._stream(k.device))
    if rc:
        _check(rc)


def lfm2sc_cache8_read(k_pages, v_pages, k_scales, v_scales, page_table, seq_len, k_out, v_out, cu_seqlens=None):
    """The values of the sequences' last tokens as rows of k_out and v_out [T, kv_heads*D] (bf16 or fp32), packed as
    lfm2sc_cache8_write takes them."""
    dev = _gpu(k_out, "k_out")
    fmt, D, H, pool = _pool8(k_pages, v_pages, k_scales, v_scales, dev)
    N, where = _table(page_table, seq_len, "seq_len", dev)
    rows, cu = _rows8(k_out, v_out, H * D, cu_seqlens, N, dev, ("k_out", "v_out"))
    rc = _lib.hybrid_lib().lfm2sc_cache8_read(_dtype_code(k_out), fmt, D, H, *pool, *where, *rows, cu, N,
                                              binding._stream(k_out.device))
    if rc:
        _check(rc)
    return k_out, v_out


def lfm2sc_attn_cached8_workspace_bytes(dtype, D, num_heads, num_kv_heads, num_seqs, L, prefix_len, max_suffix_len) -> int:
    """Never less for larger sizes: asked for with a program's largest, it serves all of its calls with the same heads."""
    code = binding._DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_lib.hybrid_lib().lfm2sc_attn_cached8_workspace_bytes(code, D, num_heads, num_kv_heads, num_seqs, L, prefix_len,
                                                                     max_suffix_len))


def lfm2sc_attn_cached8(q, k_pages, v_pages, k_scales, v_scales, prefix_pages, prefix_len, page_table, suffix_len, L, out,
                        workspace, scale=None, max_suffix_len=None):
    """lfm2sc_attn_cached over the 8-bit cache.  max_suffix_len: the caller's bound on suffix_len (None: what page_table holds);
    the workspace is asked for with the same."""
    dev = _gpu(q, "q")
    dtype = q.dtype
    fmt, D, H, pool = _pool8(k_pages, v_pages, k_scales, v_scales, dev)
    N, (table, most, lens) = _table(page_table, suffix_len, "suffix_len", dev)
    S = pool[7]
    prefix = _needed(prefix_pages, "prefix_pages", dev, _I32, -(-prefix_len // S)) if prefix_len > 0 else None
    Hq = _heads(out.shape[-1], D, "out")
    rc = _lib.hybrid_lib().lfm2sc_attn_cached8(
        _dtype_code(q), fmt, D, Hq, H, q.data_ptr(), _mat(q, "q", dev, dtype, N * L, Hq * D), N, L, *pool, prefix, prefix_len,
        table, most, lens, most * S if max_suffix_len is None else max_suffix_len, D ** -0.5 if scale is None else scale, out.data_ptr(),
        _mat(out, "out", dev, dtype, N * L, Hq * D), *_workspace(workspace, dev), binding._stream(q.device))
    if rc:
        _check(rc)
    return out
