"""Operators of the hybrid decoder's attention layers next to those of perf/operators.py, as cases that can be measured.

Three kinds of case ("op"):
  rotate  rotary positions of q and k rows, forward or gradient ("inverse")
  store   new k and v rows are quantised into a paged cache of 8 bits, and the tokens that the call touched (or the last
          "back" ones) are read back as bf16 rows
  attend  attention of new tokens (1 a sequence: decode; a block of drafts: verify) over a paged cache of 8 bits with a scale
          for each block of tokens and head, whose first `prefix` keys are shared by the whole batch

`own` False: the plain form in elementary torch operations, 32 bits (angles in 64).
`own` True: the calls a user of gated_short_causal_amd makes.

The cache: K pages [pages, kv_heads, page, dim], V pages [pages, kv_heads, page / 16, dim, 16], codes of int8 or e4m3; scales
[pages, kv_heads, page / block] fp32, a value is its code times the scale of its block of tokens.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


# ---------------------------------------------------------------- cases
# heads / kv_heads / dim: 32 / 8 / 64 is the attention of the 1.2B model whose ShortConv this library implements
# (hidden 2048); the others are generic grouped, multi-head and wide-head layouts.
def listed():
    return [
        # one user's next token: latency of a single row
        {"name": "rotate 1", "op": "rotate", "seqs": 1, "longest": 1, "lens": 1, "heads": 32, "kv_heads": 8, "dim": 64, "rotary": 64,
         "interleaved": False, "inverse": False, "packed": False, "far": 4096, "scaled": False, "type": "bf16"},
        # a packed batch of eight prompts of 64 to 2048 tokens (the library's ragged prefill workload)
        {"name": "rotate 8 x 2048 packed", "op": "rotate", "seqs": 8, "longest": 2048, "lens": 2, "heads": 32, "kv_heads": 8, "dim": 64,
         "rotary": 64, "interleaved": False, "inverse": False, "packed": True, "far": 0, "scaled": False, "type": "bf16"},
        # a long chunk far into a stretched context, half of each wide head rotated, neighbouring columns paired
        {"name": "rotate 32768 far, interleaved part", "op": "rotate", "seqs": 1, "longest": 32768, "lens": 3, "heads": 16, "kv_heads": 2,
         "dim": 128, "rotary": 64, "interleaved": True, "inverse": False, "packed": False, "far": 1 << 20, "scaled": True, "type": "bf16"},
        # training: the gradient on packed samples of odd lengths in fp32, every head with its own keys
        {"name": "rotate gradient 13 x 1531 fp32", "op": "rotate", "seqs": 13, "longest": 1531, "lens": 4, "heads": 16, "kv_heads": 16,
         "dim": 128, "rotary": 128, "interleaved": False, "inverse": True, "packed": True, "far": 0, "scaled": False, "type": "fp32"},
        # a decode step of 256 users (the library's decode batch): one token each, the block that it joins read back
        {"name": "store 256 x 1", "op": "store", "seqs": 256, "held": 600, "new": 1, "ragged": False, "back": 16, "lens": 5, "kv_heads": 8,
         "dim": 64, "page": 16, "block": 16, "codes": "e4m3"},
        # the verify workload's 64 x 8 draft tokens, long blocks
        {"name": "store 64 x 8", "op": "store", "seqs": 64, "held": 999, "new": 8, "ragged": False, "back": 72, "lens": 6, "kv_heads": 8,
         "dim": 128, "page": 64, "block": 64, "codes": "int8"},
        # eight prompts of up to 2048 tokens into an empty cache, a scale for every token
        {"name": "store 8 x 2048", "op": "store", "seqs": 8, "held": 0, "new": 2048, "ragged": True, "back": 0, "lens": 7, "kv_heads": 8,
         "dim": 64, "page": 16, "block": 1, "codes": "int8"},
        # one long document, wide heads
        {"name": "store 1 x 65536", "op": "store", "seqs": 1, "held": 0, "new": 65536, "ragged": False, "back": 0, "lens": 8, "kv_heads": 8,
         "dim": 128, "page": 128, "block": 32, "codes": "e4m3"},
        # one user, one token, a short cache: latency
        {"name": "attend 1, 500+37", "op": "attend", "seqs": 1, "new": 1, "prefix": 500, "longest": 37, "lens": 9, "heads": 32,
         "kv_heads": 8, "dim": 64, "page": 16, "block": 16, "codes": "e4m3"},
        # 256 users of one system prompt, one token each
        {"name": "attend 256, 4096+600", "op": "attend", "seqs": 256, "new": 1, "prefix": 4096, "longest": 600, "lens": 10, "heads": 32,
         "kv_heads": 8, "dim": 64, "page": 16, "block": 16, "codes": "e4m3"},
        # verify of 64 sequences x 8 draft tokens behind a long shared document
        {"name": "attend 64x8, 16384+999", "op": "attend", "seqs": 64, "new": 8, "prefix": 16384, "longest": 999, "lens": 11, "heads": 40,
         "kv_heads": 8, "dim": 128, "page": 64, "block": 64, "codes": "int8"},
        # 64 long conversations of their own, one token each, a scale for every token
        {"name": "attend 64, 16384", "op": "attend", "seqs": 64, "new": 1, "prefix": 0, "longest": 16384, "lens": 12, "heads": 24,
         "kv_heads": 8, "dim": 128, "page": 128, "block": 1, "codes": "int8"},
    ]


_HEADS = ((32, 8, 64), (16, 16, 64), (24, 8, 64), (12, 1, 64), (32, 4, 128), (16, 2, 128), (40, 8, 128), (9, 3, 128))
# rotary positions also come with head dimensions that the attention does not have
_ROTARY_HEADS = _HEADS + ((16, 4, 80), (8, 8, 96), (8, 1, 256))


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _sizes(rng):
    op = rng.choice(("rotate", "store", "attend"))
    lens = rng.randint(13, 10 ** 6)
    if op == "rotate":
        h, hkv, d = rng.choice(_ROTARY_HEADS)
        packed = rng.random() < 0.5
        return {"op": op, "seqs": _log(rng, 1, 64) if packed else 1, "longest": _log(rng, 1, 32768), "lens": lens, "heads": h, "kv_heads": hkv,
                "dim": d, "rotary": rng.choice((d, d, d // 2, 2 * rng.randint(1, d // 2))), "interleaved": rng.random() < 0.5,
                "inverse": rng.random() < 0.5, "packed": packed, "far": 0 if packed else _log(rng, 1, 1 << 24), "scaled": rng.random() < 0.5,
                "type": rng.choice(("bf16", "bf16", "fp32"))}
    page = rng.choice((16, 32, 64, 128))
    cache = {"page": page, "block": rng.choice([1] + [b for b in (16, 32, 64, 128) if b <= page]), "codes": rng.choice(("e4m3", "int8"))}
    h, hkv, d = rng.choice(_HEADS)
    if op == "store":
        new, ragged = (rng.randint(1, 8), False) if rng.random() < 0.5 else (_log(rng, 1, 65536), rng.random() < 0.5)
        return {"op": op, "seqs": _log(rng, 1, 256), "held": _log(rng, 1, 2048) if rng.random() < 0.7 else 0, "new": new, "ragged": ragged,
                "back": cache["block"] + new, "lens": lens, "kv_heads": hkv, "dim": d, **cache}
    new = rng.choice((1, 1, rng.randint(2, 8)))
    return {"op": op, "seqs": _log(rng, 1, 256), "new": new, "prefix": _log(rng, 1, 32768) if rng.random() < 0.7 else 0,
            "longest": _log(rng, new, 16384), "lens": lens, "heads": h, "kv_heads": hkv, "dim": d, **cache}


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        for key in w:
            most[c["op"], key] = max(most.get((c["op"], key), 0), w[key])
    while True:
        c = _sizes(rng)
        if c["op"] == "rotate" and c["seqs"] * c["longest"] > 65536:
            continue
        if c["op"] == "store" and c["seqs"] * (c["held"] + c["new"]) * c["kv_heads"] * c["dim"] > 65536 * 8 * 128:
            continue
        if c["op"] == "attend" and (c["seqs"] * (c["new"] * c["heads"] * (c["prefix"] + c["longest"]) + c["longest"] * c["kv_heads"] * c["dim"])
                                    > 1 << 30):
            continue
        w = work(c)
        if any(w[key] > most[c["op"], key] for key in w):
            continue
        return c


def _lengths(seed, seqs, longest, low):
    """Lengths: the longest once, the others uniform up to it; part of the case's sizes."""
    rng = random.Random(seed)
    lens = [longest] + [rng.randint(min(low, longest), longest) for _ in range(seqs - 1)]
    rng.shuffle(lens)
    return lens


def _store_lengths(case):
    """Tokens held, written and read back by sequence."""
    held = _lengths(case["lens"], case["seqs"], case["held"], 0)
    new = _lengths(case["lens"] + 1, case["seqs"], case["new"], 1) if case["ragged"] else [case["new"]] * case["seqs"]
    back = [min(h + n, case["back"]) if case["back"] else n for h, n in zip(held, new)]
    return held, new, back


def work(case):
    if case["op"] == "rotate":
        t = sum(_lengths(case["lens"], case["seqs"], case["longest"], 1))
        heads, e = case["heads"] + case["kv_heads"], 4 if case["type"] == "fp32" else 2
        return {"bytes": 2 * t * heads * case["dim"] * e + 4 * t, "flops": 3 * t * heads * case["rotary"]}
    row = 2 * case["kv_heads"] * case["dim"]                 # a token's keys and values
    if case["op"] == "store":
        held, new, back = _store_lengths(case)
        scales = 2 * case["kv_heads"] * 4 * (sum(new) + sum(back)) // case["block"]
        return {"bytes": row * 3 * (sum(new) + sum(back)) + scales, "flops": row * (2 * sum(new) + sum(back))}
    lens, n, b, p, h, d = (_lengths(case["lens"], case["seqs"], case["longest"], case["new"]), case["seqs"], case["new"], case["prefix"],
                           case["heads"], case["dim"])
    seen = sum(p * b + sum(max(0, s - b + 1 + i) for i in range(b)) for s in lens)
    keys = p + sum(lens)
    return {"bytes": row * keys + 2 * case["kv_heads"] * 4 * keys // case["block"] + 2 * n * b * h * d * 2, "flops": 4 * d * h * seen}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    return {"rotate": _prepare_rotate, "store": _prepare_store, "attend": _prepare_attend}[case["op"]](case, gen, randn)


def _prepare_rotate(case, gen, randn):
    h, hkv, d, r, dt = case["heads"], case["kv_heads"], case["dim"], case["rotary"], TYPES[case["type"]]
    lens = _lengths(case["lens"], case["seqs"], case["longest"], 1)
    t = sum(lens)
    freqs = torch.pow(10000.0, -torch.arange(0, r, 2, dtype=torch.float64) / r)
    if case["scaled"]:
        # a context eight times as long as the one that the model was trained on: slow pairs are stretched, fast ones stay
        turns = 8192 * freqs / (2 * math.pi)
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        freqs = freqs * keep + freqs / 8 * (1 - keep)
    qkv = randn(t, (h + 2 * hkv) * d).to(dt)                 # one projection's rows
    s = {"op": "rotate", "heads": h, "kv_heads": hkv, "dim": d, "rotary": r, "interleaved": case["interleaved"], "inverse": case["inverse"],
         "magnitude": 0.1 * math.log(8.0) + 1.0 if case["scaled"] else 1.0, "freqs": freqs.float().to(DEV),
         "q": qkv[:, :h * d], "k": qkv[:, h * d:(h + hkv) * d], "positions": None, "cu": None,
         "q_out": torch.empty(t, h * d, dtype=dt, device=DEV), "k_out": torch.empty(t, hkv * d, dtype=dt, device=DEV)}
    if case["packed"]:
        s["cu"] = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    else:
        first = torch.randint(0, case["far"] + 1, (1,), generator=gen, device=DEV)
        s["positions"] = (first + torch.arange(t, device=DEV)).to(torch.int32)
    return s


def _spread(randn, *shape):
    """Keys and values: channels and heads differ in size, single tokens stand out."""
    x = randn(*shape)
    return x.mul_(torch.exp(0.5 * randn(*shape[-2:]))).mul_(torch.exp(0.3 * randn(*shape[:-1], 1)))


def _power(n):
    """2^n in 32 bits, exactly, for whole n from -126 to 127."""
    return ((n.clamp(-126, 127) + 127).to(torch.int32) << 23).view(torch.float32)


def _fresh(top, codes):
    """Scale of a block whose largest magnitude is `top`."""
    if codes == "int8":
        s = top / 127
    else:
        part, power = torch.frexp(top / 448)                 # top / 448 = part * 2^power, part in [0.5, 1)
        s = _power(torch.where(part > 0.5, power, power - 1))
    return torch.where(top > 0, s.clamp(min=2.0 ** -120), 0.0)


def _code(x, codes):
    """x, in steps of its scale, as codes."""
    if codes == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _bytes(x):
    return x.view(torch.int8)


def _pool(randn, pages, case):
    """A cache full of earlier tokens: pages and scales of K and V."""
    hkv, d, page, block, codes = case["kv_heads"], case["dim"], case["page"], case["block"], case["codes"]
    got = []
    for transposed in (False, True):
        x = _spread(randn, pages, page // block, block, hkv, d)
        scale = _fresh(x.abs().amax((2, 4)), codes)          # [pages, blocks, heads]
        x = _code(x * (1 / scale)[:, :, None, :, None], codes)
        x = _bytes(x).reshape(pages, page, hkv, d).permute(0, 2, 1, 3)
        if transposed:
            x = x.reshape(pages, hkv, page // 16, 16, d).transpose(3, 4)
        got.append(x.contiguous().view(CODES[codes]))
        got.append(scale.permute(0, 2, 1).contiguous())
    return {"k_pages": got[0], "v_pages": got[2], "k_scales": got[1], "v_scales": got[3]}


def _prepare_store(case, gen, randn):
    held, new, back = _store_lengths(case)
    n, hkv, d, page = case["seqs"], case["kv_heads"], case["dim"], case["page"]
    most = max(-(-(a + b) // page) for a, b in zip(held, new))
    s = {"op": "store", "kv_heads": hkv, "dim": d, "page": page, "block": case["block"], "codes": case["codes"],
         "table": torch.randperm(n * most, generator=gen, device=DEV).to(torch.int32).reshape(n, most),
         "len": torch.tensor([a + b for a, b in zip(held, new)], dtype=torch.int32, device=DEV),
         "cu": torch.tensor([0] + new).cumsum(0).to(torch.int32).to(DEV), "ragged": case["ragged"],
         "cu_back": torch.tensor([0] + back).cumsum(0).to(torch.int32).to(DEV)}
    s.update(_pool(randn, n * most, case))
    t = sum(new)
    kv = torch.cat([_spread(randn, t, hkv, d), _spread(randn, t, hkv, d)], 1).to(torch.bfloat16).reshape(t, 2 * hkv * d)
    s.update(k=kv[:, :hkv * d], v=kv[:, hkv * d:], k_back=torch.empty(sum(back), hkv * d, dtype=torch.bfloat16, device=DEV),
             v_back=torch.empty(sum(back), hkv * d, dtype=torch.bfloat16, device=DEV))
    return s


def _prepare_attend(case, gen, randn):
    n, b, p, page, h, d = case["seqs"], case["new"], case["prefix"], case["page"], case["heads"], case["dim"]
    lens = _lengths(case["lens"], n, case["longest"], b)
    prefix_pages, most = -(-p // page), -(-max(lens) // page)
    order = torch.randperm(prefix_pages + n * most, generator=gen, device=DEV).to(torch.int32)
    s = {"op": "attend", "heads": h, "kv_heads": case["kv_heads"], "dim": d, "page": page, "block": case["block"], "new": b, "prefix": p,
         "longest": max(lens), "scale": 1.0 / math.sqrt(d), "q": randn(n * b, h * d).to(torch.bfloat16),
         "prefix_pages": order[:prefix_pages].contiguous(), "page_table": order[prefix_pages:].reshape(n, most).contiguous(),
         "suffix_len": torch.tensor(lens, dtype=torch.int32, device=DEV), "out": torch.empty(n * b, h * d, dtype=torch.bfloat16, device=DEV)}
    s.update(_pool(randn, order.numel(), case))
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _own_rotate(s):
    import gated_short_causal_amd as g
    g.lfm2sc_rotary(s["q"], s["q_out"], s["dim"], s["freqs"], positions=s["positions"], cu_seqlens=s["cu"], k=s["k"], k_out=s["k_out"],
                    interleaved=s["interleaved"], inverse=s["inverse"], magnitude=s["magnitude"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_store(s):
    import gated_short_causal_amd as g
    cache = (s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"], s["len"])
    g.lfm2sc_cache8_write(s["k"], s["v"], *cache, cu_seqlens=s["cu"] if s["ragged"] else None)
    g.lfm2sc_cache8_read(*cache, s["k_back"], s["v_back"], cu_seqlens=s["cu_back"])
    return {"k": s["k_back"], "v": s["v_back"]}


def _own_attend(s):
    import gated_short_causal_amd as g
    if "workspace" not in s:
        s["workspace"] = torch.empty(g.lfm2sc_attn_cached8_workspace_bytes(s["q"].dtype, s["dim"], s["heads"], s["kv_heads"],
                                                                           s["suffix_len"].numel(), s["new"], s["prefix"], s["longest"]),
                                     dtype=torch.uint8, device=DEV)
    g.lfm2sc_attn_cached8(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["prefix_pages"], s["prefix"], s["page_table"],
                          s["suffix_len"], s["new"], s["out"], s["workspace"], scale=s["scale"], max_suffix_len=s["longest"])
    return {"out": s["out"]}


_OWN = {"rotate": _own_rotate, "store": _own_store, "attend": _own_attend}


def _rows_of(cu, t):
    """Sequence of each packed row, and its number in it."""
    row = torch.arange(t, device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    return seq, row - cu[seq]


def _plain_rotate(s):
    t, r = s["q"].shape[0], s["rotary"]
    pos = s["positions"] if s["cu"] is None else _rows_of(s["cu"], t)[1]
    angle = pos.double()[:, None] * s["freqs"].double()      # [t, r / 2]
    cos = angle.cos().float()[:, None] * s["magnitude"]
    sin = angle.sin().float()[:, None] * (-s["magnitude"] if s["inverse"] else s["magnitude"])

    def turn(x):
        y = x.reshape(t, -1, s["dim"]).float()
        if s["interleaved"]:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :r // 2], y[..., r // 2:r]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([turned, y[..., r:]], -1).to(x.dtype).reshape(t, -1)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _places(s, cu, t):
    """Of each row of a call: page, token in the page, position in its sequence, sequence."""
    seq, local = _rows_of(cu, t)
    pos = s["len"][seq] - (cu[1:] - cu[:-1])[seq] + local
    return s["table"][seq, pos // s["page"]].long(), (pos % s["page"]).long(), pos, seq


def _plain_store(s):
    t, hkv, d, page, block, codes = s["k"].shape[0], s["kv_heads"], s["dim"], s["page"], s["block"], s["codes"]
    at, tok, _, _ = _places(s, s["cu"], t)
    start = s["len"] - (s["cu"][1:] - s["cu"][:-1])
    # the tokens before the new ones in the first block that a sequence's new ones touch
    first = start // block * block
    first_page = s["table"].gather(1, (first // page).long().clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long()
    first_block = (first % page // block).long()
    keeps = start % block > 0
    inside = first[:, None] + torch.arange(block, device=DEV)
    kept = inside < start[:, None]                                       # [n, block]
    inside = (inside % page).long()
    back_at, back_tok, _, _ = _places(s, s["cu_back"], s["k_back"].shape[0])
    limit = 127.5 if codes == "int8" else 448.0
    res = {}
    for name in ("k", "v"):
        x = s[name].float().reshape(t, hkv, d)
        pages, scales = _bytes(s[name + "_pages"]), s[name + "_scales"]
        index = (lambda p, i: (p, slice(None), i)) if name == "k" else (lambda p, i: (p, slice(None), i // 16, slice(None), i % 16))
        blocks = at * (page // block) + tok // block                     # [t]
        top = torch.zeros(scales.shape[0] * (page // block), hkv, device=DEV)
        top.scatter_reduce_(0, blocks[:, None].expand(t, hkv), x.abs().amax(-1), "amax")
        top = top.reshape(scales.shape[0], page // block, hkv).transpose(1, 2)
        touched = torch.zeros(scales.shape[0] * (page // block), dtype=torch.bool, device=DEV)
        touched[blocks] = True
        touched = touched.reshape(scales.shape[0], 1, page // block)
        has = torch.zeros_like(touched)
        has[first_page, 0, first_block] = keeps
        old = torch.where(has & touched, scales, 0.0)
        need = top * (1 / old)
        # doublings of the old scale until the new tokens fit
        part, power = torch.frexp(need / limit)
        fits = power - 1 if codes == "int8" else power - (part == 0.5).int()
        # int8: need * 2^-n < 127.5; e4m3: need * 2^-n <= 448
        n = (fits + 1 if codes == "int8" else fits).clamp(min=0)
        grown = old * _power(torch.where(old > 0, n, 0))
        scale = torch.where(touched, torch.where(old > 0, grown, _fresh(top, codes)), scales)
        # kept tokens in steps of the new scale
        seqs = torch.arange(kept.shape[0], device=DEV)[:, None].expand_as(kept)
        before = pages[index(first_page[:, None], inside)].view(CODES[codes]).float()               # [n, block, heads, d]
        ratio = (old / scale)[first_page, :, first_block]                                            # [n, heads]
        ratio = torch.where(old[first_page, :, first_block] > 0, ratio, 0.0)
        again = _bytes(_code(before * ratio[:, None, :, None], codes))
        pages[index(first_page[seqs[kept]], inside[kept])] = again[kept]
        scales.copy_(scale)
        step = scale[at, :, tok // block]                                                            # [t, heads]
        step = torch.where(step > 0, 1 / step, 0.0)
        pages[index(at, tok)] = _bytes(_code(x * step[..., None], codes))
        got = pages[index(back_at, back_tok)].view(CODES[codes]).float() * scale[back_at, :, back_tok // block][..., None]
        res[name] = got.to(torch.bfloat16).reshape(-1, hkv * d)
    return res


def _plain_attend(s):
    h, hkv, d, b, p, page, block = s["heads"], s["kv_heads"], s["dim"], s["new"], s["prefix"], s["page"], s["block"]
    n, g = s["suffix_len"].numel(), h // hkv

    def values(name, table):                                 # [..., tokens, hkv, d] of the pages of a table
        x = s[name + "_pages"][table.long()] if s[name + "_pages"].dtype == torch.int8 else \
            _bytes(s[name + "_pages"])[table.long()].view(torch.float8_e4m3fn)
        x = x.float()
        if name == "v":
            x = x.transpose(-1, -2).reshape(*table.shape, hkv, page, d)
        x = x.reshape(*table.shape, hkv, page // block, block, d) * s[name + "_scales"][table.long()][..., None, None]
        return x.reshape(*table.shape, hkv, page, d).transpose(-2, -3).reshape(*table.shape[:-1], -1, hkv, d)

    def prefix(name):    # [hkv, p, d]
        return values(name, s["prefix_pages"])[:p].permute(1, 0, 2).contiguous()

    def suffix(name):    # [n, hkv, most, d]
        return values(name, s["page_table"]).permute(0, 2, 1, 3).contiguous()

    q = s["q"].float().mul(s["scale"]).reshape(n, b, hkv, g, d)
    second = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(n, hkv, b * g, d), suffix("k").transpose(2, 3))
    most = second.shape[-1]
    second = second.reshape(n, hkv, b, g, most)
    last = s["suffix_len"][:, None].long() - b + torch.arange(b, device=DEV)       # the last own key that row (sequence, token) sees
    hidden = torch.arange(most, device=DEV) > last[:, :, None]
    score = second.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    if p:
        first = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(hkv, n * b * g, d), prefix("k").transpose(1, 2))
        score = torch.cat([first.reshape(hkv, n, b, g, p).permute(1, 0, 2, 3, 4), score], -1)
    top = score.amax(-1, keepdim=True)
    score = (score - torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    score = score / score.sum(-1, keepdim=True).clamp(min=1e-30)
    # values past a sequence's end are no values
    own_v = suffix("v").masked_fill_((torch.arange(most, device=DEV) >= s["suffix_len"][:, None])[:, None, :, None], 0.0)
    o = torch.matmul(score[..., p:].reshape(n, hkv, b * g, most), own_v).reshape(n, hkv, b, g, d)
    if p:
        o = o + torch.matmul(score[..., :p].permute(1, 0, 2, 3, 4).reshape(hkv, n * b * g, p), prefix("v")) \
            .reshape(hkv, n, b, g, d).permute(1, 0, 2, 3, 4)
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(n * b, h * d).to(torch.bfloat16)}


_PLAIN = {"rotate": _plain_rotate, "store": _plain_store, "attend": _plain_attend}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definitions in 64 bits, one sequence at a time."""
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "store": _exact_store, "attend": _exact_attend}[case["op"]](s)


def _exact_rotate(s):
    if s["cu"] is None:
        where = s["positions"].double()
    else:
        cu = s["cu"].tolist()
        where = torch.cat([torch.arange(b - a, dtype=torch.float64, device=DEV) for a, b in zip(cu, cu[1:])])
    d, r = s["dim"], s["rotary"]
    w = torch.polar(torch.full_like(where, s["magnitude"])[:, None].expand(-1, r // 2), torch.outer(where, s["freqs"].double()))
    w = w.conj() if s["inverse"] else w
    res = {}
    for name in ("q", "k"):
        x = s[name].double()
        out = x.clone()
        for head in range(x.shape[1] // d):
            c = head * d
            re, im = (slice(c, c + r, 2), slice(c + 1, c + r, 2)) if s["interleaved"] else (slice(c, c + r // 2), slice(c + r // 2, c + r))
            z = torch.complex(x[:, re].contiguous(), x[:, im].contiguous()) * w
            out[:, re], out[:, im] = z.real, z.imag
        res[name] = out
    return res


def _tokens64(pages, scales, table, transposed):
    """Codes [tokens, heads, d] and scales [tokens, heads] of the pages of one sequence."""
    x = pages.view(torch.int8)[table.long()].view(pages.dtype).double()
    if transposed:
        x = x.permute(0, 2, 4, 1, 3)                         # pages, tiles, 16, heads, d
        x = x.reshape(-1, x.shape[-2], x.shape[-1])
    else:
        x = x.permute(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])
    sc = scales[table.long()].double().permute(0, 2, 1).reshape(-1, scales.shape[1])
    return x, sc.repeat_interleave(x.shape[0] // sc.shape[0], 0)


def _power64(n):
    return ((n.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round64(x, codes):
    if codes == "int8":
        return x.round().clamp(-127, 127)
    step = _power64((torch.frexp(x).exponent - 4).clamp(min=-9))
    return ((x / step).round() * step).clamp(-448, 448)


def _exact_store(s):
    cu, back, lens = s["cu"].tolist(), s["cu_back"].tolist(), s["len"].tolist()
    block, hkv, codes = s["block"], s["kv_heads"], s["codes"]
    if len(lens) * (max(b - a for a, b in zip(cu, cu[1:])) // block + 2) > 300000:
        return None
    res = {}
    for name in ("k", "v"):
        out = torch.zeros(back[-1], hkv * s["dim"], dtype=torch.float64, device=DEV)
        for i, length in enumerate(lens):
            new = s[name][cu[i]:cu[i + 1]].double().reshape(-1, hkv, s["dim"])
            start = length - new.shape[0]
            code, old = _tokens64(s[name + "_pages"], s[name + "_scales"], s["table"][i], name == "v")
            value, old = torch.cat([code[:start] * old[:start, :, None], new]), old[:start]
            begin = start // block * block
            whole = torch.nn.functional.pad(new, (0, 0, 0, 0, start - begin, -length % block))
            top = whole.reshape(-1, block, hkv, s["dim"]).abs().amax((1, 3))        # blocks from the first touched one on
            if codes == "int8":
                scale = top / 127
            else:
                part, power = torch.frexp(top)                                      # 448 = 0.875 * 2^9
                scale = _power64(power - 9 + (part > 0.875).int())
            if start > begin:
                scale[0] = old[begin]
                for _ in range(300):
                    low = top[0] / scale[0] >= 127.5 if codes == "int8" else top[0] > 448 * scale[0]
                    scale[0] = torch.where(low, 2 * scale[0], scale[0])
            scale = scale.repeat_interleave(block, 0)[:length - begin, :, None]
            value[begin:] = _round64(value[begin:] / scale, codes) * scale
            out[back[i]:back[i + 1]] = value[length - (back[i + 1] - back[i]):length].reshape(-1, hkv * s["dim"])
        res[name] = out
    return res


def _exact_attend(s):
    h, hkv, d, b, p, g = s["heads"], s["kv_heads"], s["dim"], s["new"], s["prefix"], s["heads"] // s["kv_heads"]
    lens = s["suffix_len"].tolist()
    out = torch.zeros(len(lens) * b, h * d, dtype=torch.float64, device=DEV)

    def read(name, table, length):
        code, scale = _tokens64(s[name + "_pages"], s[name + "_scales"], table, name == "v")
        return (code * scale[..., None])[:length]

    shared = [read(name, s["prefix_pages"], p) for name in ("k", "v")] if p else None
    for i, length in enumerate(lens):
        k, v = (read(name, s["page_table"][i], length) for name in ("k", "v"))
        if p:
            k, v = torch.cat([shared[0], k]), torch.cat([shared[1], v])
        k, v = k.permute(1, 0, 2).contiguous(), v.permute(1, 0, 2).contiguous()
        q = s["q"][i * b:(i + 1) * b].double().reshape(b, hkv, g, d).permute(1, 0, 2, 3).reshape(hkv, b * g, d)
        score = (torch.matmul(q, k.transpose(1, 2).contiguous()) * s["scale"]).reshape(hkv, b, g, p + length)
        seen = p + length - b + torch.arange(b, device=DEV)
        score = score.masked_fill((torch.arange(p + length, device=DEV) > seen[:, None])[None, :, None, :], -math.inf)
        e = torch.exp(score - score.max(-1, keepdim=True).values)
        prob = (e / e.sum(-1, keepdim=True)).reshape(hkv, b * g, p + length)
        out[i * b:(i + 1) * b] = torch.matmul(prob, v).reshape(hkv, b, g, d).permute(1, 0, 2, 3).reshape(b, h * d)
    return {"out": out}
