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
from .binding import _check, _cu, _dtype_code, _i32, _ptr, _rows


def _same(ref, name, **tensors):
    _same_device_as(ref, name, **tensors)
    for n, t in tensors.items():
        if t is not None and t.dtype != ref.dtype:
            raise TypeError(f"{n} has dtype {t.dtype}; it must have {name}'s dtype {ref.dtype}")


def _same_device_as(ref, name, **tensors):
    if not binding._is_gpu(ref):
        raise ValueError(f"{name} must be a GPU tensor, got device {ref.device}")
    dev = ref.device
    for n, t in tensors.items():
        if t is not None and (not binding._is_gpu(t) or t.device != dev):
            raise ValueError(f"{n} must be on {dev} ({name}'s device), got {t.device}")


def _heads(width, D, name):
    if D <= 0 or width % D != 0:
        raise ValueError(f"{name} is {width} columns wide, not a multiple of the head dimension {D}")
    return width // D


def _f32(t, name, numel):
    if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or t.numel() < numel):
        raise ValueError(f"{name} must be a contiguous float32 tensor of at least {numel} entries")


def _workspace(t):
    if t is None:
        return None, 0
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def _prompt(q, k, v, cu_seqlens, D, out, lse, scale):
    _same(q, "q", k=k, v=v, out=out)
    _same_device_as(q, "q", cu_seqlens=cu_seqlens, lse=lse)
    T = q.shape[0]
    Hq, Hkv = _heads(out.shape[1], D, "out"), _heads(k.shape[1], D, "k")
    N = _cu(cu_seqlens)
    strides = (_rows(q, "q", T, Hq * D), _rows(k, "k", T, Hkv * D), _rows(v, "v", T, Hkv * D), _rows(out, "out", T, Hq * D))
    _f32(lse, "lse", Hq * T)
    return T, Hq, Hkv, N, strides, D ** -0.5 if scale is None else float(scale)


def lfm2sc_attn_prefill(q, k, v, cu_seqlens, D, out, lse=None, scale=None):
    """Causal attention with grouped heads over packed prompts; writes out, and lse ([heads, T] fp32) when given.
    scale defaults to D ** -0.5."""
    T, Hq, Hkv, N, (qs, ks, vs, os_), scale = _prompt(q, k, v, cu_seqlens, D, out, lse, scale)
    _check(_lib.hybrid_lib().lfm2sc_attn_prefill(
        _dtype_code(q), D, Hq, Hkv, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, cu_seqlens.data_ptr(), N,
        scale, out.data_ptr(), os_, _ptr(lse), binding._stream(q.device)))
    return out


def lfm2sc_attn_backward_workspace_bytes(dtype, D, num_heads, num_kv_heads, total_T, num_seqs) -> int:
    code = binding._DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_lib.hybrid_lib().lfm2sc_attn_backward_workspace_bytes(code, D, num_heads, num_kv_heads, total_T, num_seqs))


def lfm2sc_attn_backward(q, k, v, cu_seqlens, D, out, lse, d_out, dq, dk, dv, workspace, scale=None):
    """Backward of lfm2sc_attn_prefill: writes dq, dk and dv (summed over each group's heads)."""
    T, Hq, Hkv, N, (qs, ks, vs, os_), scale = _prompt(q, k, v, cu_seqlens, D, out, lse, scale)
    _same(q, "q", d_out=d_out, dq=dq, dk=dk, dv=dv)
    _same_device_as(q, "q", workspace=workspace)
    if lse is None:
        raise ValueError("lse of the forward is required")
    ws, ws_bytes = _workspace(workspace)
    _check(_lib.hybrid_lib().lfm2sc_attn_backward(
        _dtype_code(q), D, Hq, Hkv, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, cu_seqlens.data_ptr(), N,
        scale, out.data_ptr(), os_, lse.data_ptr(), d_out.data_ptr(), _rows(d_out, "d_out", T, Hq * D),
        dq.data_ptr(), _rows(dq, "dq", T, Hq * D), dk.data_ptr(), _rows(dk, "dk", T, Hkv * D),
        dv.data_ptr(), _rows(dv, "dv", T, Hkv * D), ws, ws_bytes, binding._stream(q.device)))
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
    if sd != 1 or (H > 1 and sh != D):
        raise ValueError(f"{name}: a token's heads must be dense, got strides {t.stride()}")
    if S == 1:
        st = sp if P > 1 else H * D
    if P > 1 and sp != S * st:
        raise ValueError(f"{name}: pages must be {S} token strides apart, got strides {t.stride()}")
    return P, S, H, D, st


def lfm2sc_attn_cached(q, k_pages, v_pages, prefix_pages, prefix_len, page_table, suffix_len, L, out, workspace,
                       scale=None):
    """Attention of L new tokens per sequence (q [N*L, heads*D], the rows of a verify block; L = 1: decode) over a paged
    cache: the prefix_len keys of prefix_pages, shared by the batch, then each sequence's own suffix_len keys (the new ones
    included) in its page_table row [N, max_pages]."""
    P, S, Hkv, D, stride = _pages(k_pages, "k_pages")
    if _pages(v_pages, "v_pages") != (P, S, Hkv, D, stride):
        raise ValueError("k_pages and v_pages must have the same shape and strides")
    _same(q, "q", k_pages=k_pages, v_pages=v_pages, out=out)
    _same_device_as(q, "q", prefix_pages=prefix_pages, page_table=page_table, suffix_len=suffix_len, workspace=workspace)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [N, max_pages]")
    N, most = page_table.shape
    _i32(page_table, "page_table")
    _i32(suffix_len, "suffix_len", N)
    if prefix_len > 0:
        if prefix_pages is None:
            raise ValueError("prefix_pages is required with a prefix")
        _i32(prefix_pages, "prefix_pages", -(-prefix_len // S))
    Hq = _heads(out.shape[1], D, "out")
    qs, os_ = _rows(q, "q", N * L, Hq * D), _rows(out, "out", N * L, Hq * D)
    ws, ws_bytes = _workspace(workspace)
    _check(_lib.hybrid_lib().lfm2sc_attn_cached(
        _dtype_code(q), D, Hq, Hkv, q.data_ptr(), qs, N, L, k_pages.data_ptr(), v_pages.data_ptr(), stride, P, S,
        _ptr(prefix_pages), prefix_len, page_table.data_ptr(), most, suffix_len.data_ptr(),
        D ** -0.5 if scale is None else float(scale), out.data_ptr(), os_, ws, ws_bytes, binding._stream(q.device)))
    return out


def lfm2sc_accept_drafts_workspace_bytes(num_seqs, L, V) -> int:
    return int(_lib.hybrid_lib().lfm2sc_accept_drafts_workspace_bytes(num_seqs, L, V))


def lfm2sc_accept_drafts(target_probs, draft_tokens, u_accept, u_sample, accept_len, next_token, workspace,
                         draft_probs=None, num_drafts=None, keep_len=None):
    """Speculative verification: accept_len [N] drafts of draft_tokens [N, L] are kept, next_token [N] is drawn from what
    is left; keep_len [N] = accept_len + 1 is the accept length lfm2sc_commit_window takes for a block that starts with
    the last sampled token.  u_accept [N, L], u_sample [N]: uniform fp32 numbers in [0, 1)."""
    if draft_tokens.dim() != 2:
        raise ValueError("draft_tokens must be [N, L]")
    N, L = draft_tokens.shape
    if target_probs.dim() != 2:
        raise ValueError("target_probs must be [N*(L+1), V]")
    V = target_probs.shape[1]
    _same(target_probs, "target_probs", draft_probs=draft_probs)
    _same_device_as(target_probs, "target_probs", draft_tokens=draft_tokens, u_accept=u_accept, u_sample=u_sample,
                    accept_len=accept_len, next_token=next_token, workspace=workspace, num_drafts=num_drafts,
                    keep_len=keep_len)
    ts = max(V, _rows(target_probs, "target_probs", N * (L + 1), V))
    ds = 0 if draft_probs is None else max(V, _rows(draft_probs, "draft_probs", N * L, V))
    _i32(draft_tokens, "draft_tokens")
    for name, t in (("accept_len", accept_len), ("next_token", next_token), ("num_drafts", num_drafts),
                    ("keep_len", keep_len)):
        _i32(t, name, N)
    _f32(u_accept, "u_accept", N * L)
    _f32(u_sample, "u_sample", N)
    ws, ws_bytes = _workspace(workspace)
    _check(_lib.hybrid_lib().lfm2sc_accept_drafts(
        _dtype_code(target_probs), V, N, L, target_probs.data_ptr(), ts, _ptr(draft_probs), ds, draft_tokens.data_ptr(),
        _ptr(num_drafts), u_accept.data_ptr(), u_sample.data_ptr(), accept_len.data_ptr(), _ptr(keep_len),
        next_token.data_ptr(), ws, ws_bytes, binding._stream(target_probs.device)))
    return accept_len, next_token
