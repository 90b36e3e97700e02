"""Python binding of include/lfm2sc_hybrid.h: attention over packed prompts and over a paged cache, and draft
verification, in the manner of ``binding``: the C entry points' names, torch tensors in, caller-owned outputs
written in place on the current stream, and checks of everything visible in the tensors before any library call.

Tensor conventions (see the header for the full contract):
  q, out, gradients  [rows, >= heads*D]  bf16, unit column stride; the number of heads is the width over D
  k, v               [rows, kv_heads*D]
  k_pages, v_pages   [pages, page_size, kv_heads, D] bf16, the last two dense, pages evenly spaced
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
