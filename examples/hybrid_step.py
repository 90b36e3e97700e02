"""The hybrid decoder's operators as a program uses them: one training step of a ShortConv layer and an attention layer,
one speculative serving step (verify block through both kinds of layer, draft verification, rollback of the conv
states), and decoding over a cache of 8-bit codes.  Sizes: hidden 2048, K = 3, 32 query and 8 key/value heads of 64.  Random weights; `python examples/hybrid_step.py`
on an MI355X.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_short_causal_amd as g  # noqa: E402

H, K, HEADS, KV, D = 2048, 3, 32, 8, 64
BF, I32 = torch.bfloat16, torch.int32


def rand(*shape, dev, scale=1.0):
    return (torch.randn(*shape, device=dev) * scale).to(BF)


def train_step(lens, dev):
    """Forward and backward of both layers over packed sequences; returns outputs and gradients."""
    T, N = sum(lens), len(lens)
    cu = torch.tensor([0] + lens).cumsum(0).to(I32).to(dev)
    conv_in, w, dy = rand(T, 3 * H, dev=dev), rand(H, K, dev=dev, scale=0.3), rand(T, H, dev=dev)
    y, d_conv, dw = torch.empty_like(dy), torch.empty_like(conv_in), torch.empty(H, K, device=dev)
    ws = torch.empty(g.lfm2sc_backward_workspace_bytes(BF, H, K, T, N), dtype=torch.uint8, device=dev)
    g.lfm2sc_prefill_ragged(conv_in, cu, w, y)
    g.lfm2sc_backward(conv_in, cu, w, dy, d_conv, dw, ws)

    # k and v are columns of one projection's rows, their gradients columns of one buffer
    q, kv, do = rand(T, HEADS * D, dev=dev), rand(T, 2 * KV * D, dev=dev), rand(T, HEADS * D, dev=dev)
    out, lse, dq, d_kv = torch.empty_like(q), torch.empty(HEADS, T, device=dev), torch.empty_like(q), torch.empty_like(kv)
    k, v = kv.split(KV * D, 1)
    dk, dv = d_kv.split(KV * D, 1)
    ws = torch.empty(g.lfm2sc_attn_backward_workspace_bytes(BF, D, HEADS, KV, T, N), dtype=torch.uint8, device=dev)
    freqs = g.lfm2sc_rotary_freqs(D, base=1e6).to(dev)
    g.lfm2sc_rotary(q, q, D, freqs, cu_seqlens=cu, k=k, k_out=k)
    g.lfm2sc_attn_prefill(q, k, v, cu, D, out, lse=lse)
    g.lfm2sc_attn_backward(q, k, v, cu, D, out, lse, do, dq, dk, dv, ws)
    g.lfm2sc_rotary(dq, dq, D, freqs, cu_seqlens=cu, k=dk, k_out=dk, inverse=True)
    return {"y": y, "d_conv": d_conv, "dw": dw, "out": out, "lse": lse, "dq": dq, "d_kv": d_kv}


def speculative_step(seqs, drafts, prefix, dev, vocab=4096, page=16):
    """A block of the last sampled token and `drafts` drafted ones per sequence; returns the tokens kept and the next one."""
    L = drafts + 1
    # ShortConv layer: the block from the slots' states, every state on the tape
    slots = torch.randperm(2 * seqs, device=dev)[:seqs].to(I32)
    pool, w = rand(2 * seqs, H, K, dev=dev), rand(H, K, dev=dev, scale=0.3)
    tape, y = torch.empty(seqs, L, H, K, dtype=BF, device=dev), torch.empty(seqs * L, H, dtype=BF, device=dev)
    g.lfm2sc_verify_window(rand(seqs * L, 3 * H, dev=dev), w, pool, slots, L, tape, y)

    # attention layer: the block's keys and values are in the sequences' pages already
    lens = torch.randint(L, 200, (seqs,), device=dev).to(I32)
    most, shared = -(-200 // page), -(-prefix // page)
    cache = rand(shared + seqs * most, page, 2, KV, D, dev=dev)
    pages = torch.randperm(cache.shape[0], device=dev).to(I32)
    table = pages[shared:].reshape(seqs, most).contiguous()
    out = torch.empty(seqs * L, HEADS * D, dtype=BF, device=dev)
    ws = torch.empty(g.lfm2sc_attn_cached_workspace_bytes(BF, D, HEADS, KV, seqs, L, prefix, most, page), dtype=torch.uint8,
                     device=dev)
    g.lfm2sc_attn_cached(rand(seqs * L, HEADS * D, dev=dev), cache[:, :, 0], cache[:, :, 1], pages[:shared].contiguous(), prefix,
                         table, lens, L, out, ws)

    # the target's and the drafter's probabilities, then the accept boundary and the conv states at it
    logits = torch.randn(seqs, L, vocab, device=dev) * 2
    target = torch.softmax(logits, -1).reshape(seqs * L, vocab)
    draft = torch.softmax(logits[:, :drafts] + 0.5 * torch.randn(seqs, drafts, vocab, device=dev), -1).reshape(-1, vocab)
    tokens = torch.multinomial(draft, 1).reshape(seqs, drafts).to(I32)
    accepted, keep, following = (torch.empty(seqs, dtype=I32, device=dev) for _ in range(3))
    ws = torch.empty(g.lfm2sc_accept_drafts_workspace_bytes(seqs, drafts, vocab), dtype=torch.uint8, device=dev)
    g.lfm2sc_accept_drafts(target, tokens, torch.rand(seqs, drafts, device=dev), torch.rand(seqs, device=dev), accepted, following,
                           ws, draft_probs=draft, keep_len=keep)
    g.lfm2sc_commit_window(tape, keep, pool, slots)
    return {"y": y, "out": out, "accepted": accepted, "next": following, "pool": pool, "tape": tape, "slots": slots}


def decode_8bit(prompts, steps, prefix, dev, page=64, block=16, codes=torch.float8_e4m3fn):
    """Attention layer of `steps` decode steps over a cache of 8-bit codes: a shared prefix and prompts of their own are
    written once, then each step rotates, writes and attends one token per sequence; returns the steps' outputs."""
    N, limit = len(prompts), max(prompts) + steps
    most, shared = -(-limit // page), -(-prefix // page)
    P = shared + N * most
    k_pages, v_pages = (torch.empty(P, KV, *shape, dtype=codes, device=dev) for shape in ((page, D), (page // 16, D, 16)))
    k_scales, v_scales = (torch.empty(P, KV, page // block, device=dev) for _ in range(2))
    cache = (k_pages, v_pages, k_scales, v_scales)
    pages = torch.randperm(P, device=dev).to(I32)
    prefix_pages, table = pages[:shared].contiguous(), pages[shared:].reshape(N, most).contiguous()
    freqs = g.lfm2sc_rotary_freqs(D, base=1e6).to(dev)

    def rotated(rows, **where):
        q, k, v = rows.split([HEADS * D, KV * D, KV * D], 1)             # one projection's columns, rotated in place
        g.lfm2sc_rotary(q, q, D, freqs, k=k, k_out=k, **where)
        return q, k, v

    width = (HEADS + 2 * KV) * D
    zero, one = torch.tensor([0, prefix], dtype=I32, device=dev), torch.tensor([prefix], dtype=I32, device=dev)
    _, k, v = rotated(rand(prefix, width, dev=dev), cu_seqlens=zero)
    g.lfm2sc_cache8_write(k, v, *cache, prefix_pages[None], one)
    lens = torch.tensor(prompts, dtype=I32, device=dev)
    cu = torch.tensor([0] + prompts).cumsum(0).to(I32).to(dev)
    _, k, v = rotated(rand(sum(prompts), width, dev=dev), cu_seqlens=cu, positions=torch.full((N,), prefix, dtype=I32, device=dev))
    g.lfm2sc_cache8_write(k, v, *cache, table, lens, cu_seqlens=cu)

    ws = torch.empty(g.lfm2sc_attn_cached8_workspace_bytes(BF, D, HEADS, KV, N, 1, prefix, limit), dtype=torch.uint8, device=dev)
    outs = []
    for _ in range(steps):
        q, k, v = rotated(rand(N, width, dev=dev), positions=lens + prefix)
        lens += 1
        g.lfm2sc_cache8_write(k, v, *cache, table, lens)
        outs.append(torch.empty(N, HEADS * D, dtype=BF, device=dev))
        g.lfm2sc_attn_cached8(q, *cache, prefix_pages, prefix, table, lens, 1, outs[-1], ws, max_suffix_len=limit)
    return {"out": torch.stack(outs), "lens": lens, "cache": cache, "table": table, "prefix_pages": prefix_pages}


if __name__ == "__main__":
    device = torch.device("cuda:0")
    grads = train_step([700, 1, 323], device)
    print("training step:", {k: tuple(v.shape) for k, v in grads.items()})
    step = speculative_step(16, 7, 1000, device)
    torch.cuda.synchronize()
    print("speculative step: accepted", step["accepted"].tolist(), "next", step["next"].tolist())
    decoded = decode_8bit([100, 7, 333], 4, 500, device)
    print("8-bit decoding:", tuple(decoded["out"].shape), "lengths", decoded["lens"].tolist())
