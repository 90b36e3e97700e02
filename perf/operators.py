"""Operators of the hybrid decoder around the ShortConv, as cases that can be measured.

Four kinds of case ("op"):
  prompt  causal attention with grouped heads over packed sequences of different lengths (serving: output and lse)
  train   the same forward and its backward (output, lse, dq, dk, dv)
  cached  attention of new tokens (1 a sequence: decode; a block of drafts: verify) over a paged cache whose first
          `prefix` keys are shared by the whole batch
  drafts  verification of drafted tokens against the target's probabilities, from given random numbers

`own` False: the plain form in elementary torch operations, 32 bits (64 for the sums the drafts' choice hangs on).
`own` True: the calls a user of gated_short_causal_amd makes.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases
# heads / kv_heads / dim: 32 / 8 / 64 is the attention of the 1.2B model whose ShortConv this library implements
# (hidden 2048); the others are generic grouped, multi-head and wide-head layouts.
def listed():
    return [
        # one short question: latency of a single small prompt
        {"name": "prompt 1 x 48", "op": "prompt", "seqs": 1, "longest": 48, "lens": 1, "heads": 32, "kv_heads": 8, "dim": 64},
        # a packed batch of eight prompts of 64 to 2048 tokens (the library's ragged prefill workload)
        {"name": "prompt 8 x 2048", "op": "prompt", "seqs": 8, "longest": 2048, "lens": 2, "heads": 32, "kv_heads": 8, "dim": 64},
        # one long document, wide heads, few kv heads
        {"name": "prompt 1 x 8192 wide", "op": "prompt", "seqs": 1, "longest": 8192, "lens": 3, "heads": 16, "kv_heads": 2, "dim": 128},
        # fine-tuning on packed samples of odd lengths, every head with its own keys
        {"name": "train 13 x 1531 wide", "op": "train", "seqs": 13, "longest": 1531, "lens": 4, "heads": 16, "kv_heads": 16, "dim": 128},
        # the library's shorter training length
        {"name": "train 1 x 4096", "op": "train", "seqs": 1, "longest": 4096, "lens": 5, "heads": 32, "kv_heads": 8, "dim": 64},
        # long-context training
        {"name": "train 1 x 8192", "op": "train", "seqs": 1, "longest": 8192, "lens": 6, "heads": 32, "kv_heads": 8, "dim": 64},
        # one user, one token, a short cache: latency
        {"name": "decode 1, 500+37", "op": "cached", "seqs": 1, "block": 1, "prefix": 500, "longest": 37, "lens": 7, "heads": 32,
         "kv_heads": 8, "dim": 64, "page": 16},
        # 256 users of one system prompt, one token each (the library's decode batch)
        {"name": "decode 256, 4096+600", "op": "cached", "seqs": 256, "block": 1, "prefix": 4096, "longest": 600, "lens": 8, "heads": 32,
         "kv_heads": 8, "dim": 64, "page": 16},
        # verify of 64 sequences x 8 draft tokens (the library's verify workload) behind a long shared document
        {"name": "verify 64x8, 16384+999", "op": "cached", "seqs": 64, "block": 8, "prefix": 16384, "longest": 999, "lens": 9, "heads": 40,
         "kv_heads": 8, "dim": 128, "page": 64},
        # one user, four drafts, odd vocabulary: latency
        {"name": "drafts 1x4, 32003", "op": "drafts", "seqs": 1, "block": 4, "vocab": 32003, "type": "fp32", "draft_rows": True},
        # 64 sequences, a verify block of 8 tokens = 7 drafts and the last token
        {"name": "drafts 64x7, 65536", "op": "drafts", "seqs": 64, "block": 7, "vocab": 65536, "type": "fp32", "draft_rows": True},
        # a full batch with greedy drafts (no draft probabilities) and bf16 rows of a large vocabulary
        {"name": "drafts 256x7, 128256", "op": "drafts", "seqs": 256, "block": 7, "vocab": 128256, "type": "bf16", "draft_rows": False},
    ]


_HEADS = ((32, 8, 64), (16, 16, 64), (24, 8, 64), (12, 1, 64), (32, 4, 128), (16, 2, 128), (40, 8, 128), (9, 3, 128))


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _sizes(rng):
    op = rng.choice(("prompt", "train", "cached", "drafts"))
    if op == "drafts":
        return {"op": op, "seqs": _log(rng, 1, 256), "block": rng.randint(1, 8), "vocab": _log(rng, 1000, 160000),
                "type": rng.choice(("fp32", "bf16")), "draft_rows": rng.random() < 0.7}
    h, hkv, d = rng.choice(_HEADS)
    heads = {"heads": h, "kv_heads": hkv, "dim": d, "lens": rng.randint(10, 10 ** 6)}
    if op == "cached":
        block = rng.choice((1, 1, rng.randint(2, 8)))
        return {"op": op, "seqs": _log(rng, 1, 256), "block": block, "prefix": _log(rng, 1, 32768) if rng.random() < 0.9 else 0,
                "longest": _log(rng, block, 2048), "page": rng.choice((16, 32, 64, 128)), **heads}
    return {"op": op, "seqs": _log(rng, 1, 64), "longest": _log(rng, 1, 8192), **heads}


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        for key in w:
            most[c["op"], key] = max(most.get((c["op"], key), 0), w[key])
    while True:
        c = _sizes(rng)
        w = work(c)
        if any(w[key] > most[c["op"], key] for key in w):
            continue
        if c["op"] == "drafts" and c["seqs"] * (c["block"] + 1) * c["vocab"] > 256 * 8 * 128256:
            continue
        if c["op"] in ("prompt", "train") and c["seqs"] * c["longest"] ** 2 > 8192 ** 2:
            continue
        if c["op"] == "cached" and c["seqs"] * (c["block"] * c["heads"] * (c["prefix"] + c["longest"]) + c["longest"] * c["kv_heads"] * c["dim"]) > 1 << 30:
            continue
        return c


def _lengths(case):
    """Sequence lengths: the longest once, the others uniform up to it; part of the case's sizes."""
    rng = random.Random(case["lens"])
    low = case.get("block", 1)
    lens = [case["longest"]] + [rng.randint(low, case["longest"]) for _ in range(case["seqs"] - 1)]
    rng.shuffle(lens)
    return lens


def work(case):
    if case["op"] == "drafts":
        # one row of the target's and one of the drafts' probabilities a sequence, and the drafts' own numbers
        n, e = case["seqs"], 4 if case["type"] == "fp32" else 2
        rows = 2 if case["draft_rows"] else 1
        return {"bytes": n * (case["vocab"] * e * rows + case["block"] * (8 + e * rows) + 12), "flops": 2 * n * case["vocab"] * rows}
    lens, h, hkv, d = _lengths(case), case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "cached":
        n, b, p = case["seqs"], case["block"], case["prefix"]
        seen = sum(p * b + sum(max(0, s - b + 1 + i) for i in range(b)) for s in lens)
        return {"bytes": 2 * hkv * d * 2 * (p + sum(lens)) + 2 * n * b * h * d * 2, "flops": 4 * d * h * seen}
    t, pairs = sum(lens), sum(s * (s + 1) // 2 for s in lens)
    fwd = {"bytes": t * (2 * h + 2 * hkv) * d * 2 + t * h * 4, "flops": 4 * d * h * pairs}
    if case["op"] == "prompt":
        return fwd
    # the backward: five products, q k v out dout read, dq dk dv written
    return {"bytes": fwd["bytes"] + t * (4 * h + 4 * hkv) * d * 2 + t * h * 4, "flops": fwd["flops"] + 10 * d * h * pairs}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    if case["op"] == "drafts":
        return _prepare_drafts(case, gen, randn)
    lens, h, hkv, d = _lengths(case), case["heads"], case["kv_heads"], case["dim"]
    s = {"op": case["op"], "heads": h, "kv_heads": hkv, "dim": d, "scale": 1.0 / math.sqrt(d)}
    if case["op"] == "cached":
        n, b, p, page = case["seqs"], case["block"], case["prefix"], case["page"]
        prefix_pages, most = -(-p // page), -(-max(lens) // page)
        pages = prefix_pages + n * most
        order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
        s.update(block=b, prefix=p, q=randn(n * b, h * d).to(torch.bfloat16),
                 k_pages=randn(pages, page, hkv, d).to(torch.bfloat16), v_pages=randn(pages, page, hkv, d).to(torch.bfloat16),
                 prefix_pages=order[:prefix_pages].contiguous(), page_table=order[prefix_pages:].reshape(n, most).contiguous(),
                 suffix_len=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 out=torch.empty(n * b, h * d, dtype=torch.bfloat16, device=DEV))
        return s
    t = sum(lens)
    cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)
    # k and v are columns of one projection's output rows
    q, kv = randn(t, h * d).to(torch.bfloat16), randn(t, 2 * hkv * d).to(torch.bfloat16)
    s.update(q=q, k=kv[:, :hkv * d], v=kv[:, hkv * d:], cu=cu.to(DEV), longest=max(lens),
             out=torch.empty(t, h * d, dtype=torch.bfloat16, device=DEV), lse=torch.empty(h, t, dtype=torch.float32, device=DEV))
    if case["op"] == "train":
        d_kv = torch.empty_like(kv)
        s.update(d_out=randn(t, h * d).to(torch.bfloat16), dq=torch.empty_like(q), dk=d_kv[:, :hkv * d], dv=d_kv[:, hkv * d:])
    return s


def _prepare_drafts(case, gen, randn):
    """Peaked rows as a language model gives them; the draft model's logits are the target's with noise."""
    n, b, v = case["seqs"], case["block"], case["vocab"]
    dt = torch.float32 if case["type"] == "fp32" else torch.bfloat16
    logits = randn(n, b + 1, v).mul_(2.5)
    target = torch.softmax(logits, -1).to(dt).reshape(n * (b + 1), v)
    logits = logits[:, :b]
    logits = logits + 0.7 * randn(n, b, v)
    if case["draft_rows"]:
        draft = torch.softmax(logits, -1)
        tokens = torch.multinomial(draft.reshape(n * b, v), 1, generator=gen).reshape(n, b)
        draft = draft.to(dt).reshape(n * b, v)
    else:
        draft, tokens = None, logits.argmax(-1)
    return {"op": "drafts", "target": target, "draft": draft, "tokens": tokens.to(torch.int32).contiguous(),
            "u_accept": torch.rand(n, b, generator=gen, device=DEV), "u_sample": torch.rand(n, generator=gen, device=DEV),
            "accept_len": torch.empty(n, dtype=torch.int32, device=DEV), "keep_len": torch.empty(n, dtype=torch.int32, device=DEV),
            "next_token": torch.empty(n, dtype=torch.int32, device=DEV)}


# ---------------------------------------------------------------- one pass
def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _own_prompt(s):
    import gated_short_causal_amd as g
    g.lfm2sc_attn_prefill(s["q"], s["k"], s["v"], s["cu"], s["dim"], s["out"], lse=s["lse"], scale=s["scale"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_train(s):
    import gated_short_causal_amd as g
    if "workspace" not in s:
        s["workspace"] = torch.empty(g.lfm2sc_attn_backward_workspace_bytes(s["q"].dtype, s["dim"], s["heads"], s["kv_heads"],
                                                                            s["q"].shape[0], s["cu"].numel() - 1), dtype=torch.uint8, device=DEV)
    g.lfm2sc_attn_prefill(s["q"], s["k"], s["v"], s["cu"], s["dim"], s["out"], lse=s["lse"], scale=s["scale"])
    g.lfm2sc_attn_backward(s["q"], s["k"], s["v"], s["cu"], s["dim"], s["out"], s["lse"], s["d_out"], s["dq"], s["dk"], s["dv"], s["workspace"],
                           scale=s["scale"])
    return {k: s[k] for k in ("out", "lse", "dq", "dk", "dv")}


def _own_cached(s):
    import gated_short_causal_amd as g
    if "workspace" not in s:
        s["workspace"] = torch.empty(g.lfm2sc_attn_cached_workspace_bytes(s["q"].dtype, s["dim"], s["heads"], s["kv_heads"], s["suffix_len"].numel(),
                                                                          s["block"], s["prefix"], s["page_table"].shape[1], s["k_pages"].shape[1]),
                                     dtype=torch.uint8, device=DEV)
    g.lfm2sc_attn_cached(s["q"], s["k_pages"], s["v_pages"], s["prefix_pages"], s["prefix"], s["page_table"], s["suffix_len"], s["block"], s["out"],
                         s["workspace"], scale=s["scale"])
    return {"out": s["out"]}


def _own_drafts(s):
    import gated_short_causal_amd as g
    if "workspace" not in s:
        s["workspace"] = torch.empty(g.lfm2sc_accept_drafts_workspace_bytes(s["tokens"].shape[0], s["tokens"].shape[1], s["target"].shape[1]),
                                     dtype=torch.uint8, device=DEV)
    g.lfm2sc_accept_drafts(s["target"], s["tokens"], s["u_accept"], s["u_sample"], s["accept_len"], s["next_token"], s["workspace"],
                           draft_probs=s["draft"], keep_len=s["keep_len"])
    return {k: s[k] for k in ("accept_len", "keep_len", "next_token")}


_OWN = {"prompt": _own_prompt, "train": _own_train, "cached": _own_cached, "drafts": _own_drafts}


def _padded(s):
    """The packed rows as [sequence, position, ...] with the sequence and position of every packed row, all on the device."""
    t, cu, longest = s["q"].shape[0], s["cu"].long(), s["longest"]
    row = torch.arange(t, device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    pos = torch.arange(longest, device=DEV)
    index = (cu[:-1, None] + pos).clamp(max=t - 1)
    here = pos < (cu[1:] - cu[:-1])[:, None]
    return seq, row - cu[seq], index, here


def _plain_prompt(s):
    return _plain_attention(s, False)


def _plain_train(s):
    return _plain_attention(s, True)


def _plain_attention(s, backward):
    h, hkv, d, longest = s["heads"], s["kv_heads"], s["dim"], s["longest"]
    g = h // hkv
    seq, at, index, here = _padded(s)
    n = index.shape[0]

    def queries(x):   # [n, hkv, g * longest, d]
        return x[index].float().reshape(n, longest, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * longest, d)

    def keys(x):      # [n, hkv, longest, d]
        return x[index].float().reshape(n, longest, hkv, d).permute(0, 2, 1, 3).contiguous()

    def rows(x):      # [n, hkv, g, longest, ...] back to packed rows
        return x.permute(0, 3, 1, 2, *range(4, x.dim()))[seq, at]

    q, k, v = queries(s["q"]), keys(s["k"]), keys(s["v"])
    pos = torch.arange(longest, device=DEV)
    hidden = (pos[None, :] > pos[:, None])[None, None, None] | ~here[:, None, None, None, :]
    p = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).reshape(n, hkv, g, longest, longest)
    p.masked_fill_(hidden, -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    p.div_(total)
    p = p.reshape(n, hkv, g * longest, longest)
    o = torch.matmul(p, v)
    t = s["q"].shape[0]
    res = {"out": rows(o.reshape(n, hkv, g, longest, d)).reshape(t, h * d).to(torch.bfloat16), "lse": rows(lse).reshape(t, h).t().contiguous()}
    if not backward:
        return res
    # rows of the padding carry no gradient
    do = queries(s["d_out"]).reshape(n, hkv, g, longest, d).mul_(here[:, None, None, :, None]).reshape(n, hkv, g * longest, d)
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    del p
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3), q)
    res["dq"] = rows(dq.reshape(n, hkv, g, longest, d)).reshape(t, h * d).to(torch.bfloat16)
    res["dk"] = dk.permute(0, 2, 1, 3)[seq, at].reshape(t, hkv * d).to(torch.bfloat16)
    res["dv"] = dv.permute(0, 2, 1, 3)[seq, at].reshape(t, hkv * d).to(torch.bfloat16)
    return res


def _plain_cached(s):
    h, hkv, d, b, p = s["heads"], s["kv_heads"], s["dim"], s["block"], s["prefix"]
    n, g = s["suffix_len"].numel(), h // hkv

    def prefix(x):    # [hkv, p, d]
        return x[s["prefix_pages"].long()].reshape(-1, hkv, d)[:p].float().permute(1, 0, 2).contiguous()

    def suffix(x):    # [n, hkv, most, d]
        return x[s["page_table"].long()].reshape(n, -1, hkv, d).float().permute(0, 2, 1, 3).contiguous()

    q = s["q"].float().mul(s["scale"]).reshape(n, b, hkv, g, d)
    kp, ks = prefix(s["k_pages"]), suffix(s["k_pages"])
    most = ks.shape[2]
    first = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(hkv, n * b * g, d), kp.transpose(1, 2))
    first = first.reshape(hkv, n, b, g, p).permute(1, 0, 2, 3, 4)
    second = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(n, hkv, b * g, d), ks.transpose(2, 3)).reshape(n, hkv, b, g, most)
    last = s["suffix_len"][:, None].long() - b + torch.arange(b, device=DEV)       # the last own key that row (sequence, draft) sees
    hidden = torch.arange(most, device=DEV) > last[:, :, None]
    score = torch.cat([first, second.masked_fill(hidden[:, None, :, None, :], -math.inf)], -1)
    top = score.amax(-1, keepdim=True)
    score = (score - torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    score = score / score.sum(-1, keepdim=True).clamp(min=1e-30)
    vp, vs = prefix(s["v_pages"]), suffix(s["v_pages"])
    o = torch.matmul(score[..., :p].permute(1, 0, 2, 3, 4).reshape(hkv, n * b * g, p), vp).reshape(hkv, n, b, g, d).permute(1, 0, 2, 3, 4)
    o = o + torch.matmul(score[..., p:].reshape(n, hkv, b * g, most), vs).reshape(n, hkv, b, g, d)
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(n * b, h * d).to(torch.bfloat16)}


def _plain_drafts(s):
    tokens, u = s["tokens"].long(), s["u_accept"].double()
    n, b = tokens.shape
    target = s["target"].reshape(n, b + 1, -1)
    v = target.shape[2]
    p = target[:, :b].gather(2, tokens[..., None]).squeeze(2).double()
    if s["draft"] is not None:
        draft = s["draft"].reshape(n, b, v)
        q = draft.gather(2, tokens[..., None]).squeeze(2).double()
    else:
        q = torch.ones_like(p)
    accepted = (u * q < p).long().cumprod(1).sum(1)
    every, seq = torch.arange(v, device=DEV), torch.arange(n, device=DEV)
    row = target[seq, accepted].double()
    at = accepted.clamp(max=b - 1)
    if s["draft"] is not None:
        less = (row - draft[seq, at].double()).clamp(min=0)
    else:
        less = torch.where(every == tokens[seq, at][:, None], 0.0, row)
    rest = torch.where((accepted < b)[:, None], less, row)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, row)
    cum = rest.cumsum(1)
    after = (cum <= s["u_sample"].double()[:, None] * cum[:, -1:]).sum(1)
    return {"accept_len": accepted.to(torch.int32), "keep_len": (accepted + 1).to(torch.int32), "next_token": after.to(torch.int32)}


_PLAIN = {"prompt": _plain_prompt, "train": _plain_train, "cached": _plain_cached, "drafts": _plain_drafts}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definitions in 64 bits, one sequence and one group of heads at a time.  The drafts' outputs are whole numbers: no value."""
    if case["op"] == "drafts":
        return None
    s = prepare(case, seed)
    return _exact_cached(s) if case["op"] == "cached" else _exact_attention(s, case["op"] == "train")


def _softmax64(score):
    top = score.max(-1, keepdim=True).values
    e = torch.exp(score - top)
    z = e.sum(-1, keepdim=True)
    return e / z, (top + torch.log(z))[..., 0]


def _exact_attention(s, backward):
    h, hkv, d, g = s["heads"], s["kv_heads"], s["dim"], s["heads"] // s["kv_heads"]
    cu = s["cu"].tolist()
    t = cu[-1]
    res = {"out": torch.zeros(t, h * d, dtype=torch.float64, device=DEV), "lse": torch.zeros(h, t, dtype=torch.float64, device=DEV)}
    if backward:
        res.update(dq=torch.zeros(t, h * d, dtype=torch.float64, device=DEV), dk=torch.zeros(t, hkv * d, dtype=torch.float64, device=DEV),
                   dv=torch.zeros(t, hkv * d, dtype=torch.float64, device=DEV))
    for a, b in zip(cu, cu[1:]):
        future = torch.ones(b - a, b - a, dtype=torch.bool, device=DEV).triu(1)
        for head in range(h):
            col, kcol = slice(head * d, (head + 1) * d), slice(head // g * d, (head // g + 1) * d)
            q, k, v = s["q"][a:b, col].double(), s["k"][a:b, kcol].double(), s["v"][a:b, kcol].double()
            prob, lse = _softmax64((q @ k.t() * s["scale"]).masked_fill(future, -math.inf))
            o = prob @ v
            res["out"][a:b, col] = o
            res["lse"][head, a:b] = lse
            if backward:
                do = s["d_out"][a:b, col].double()
                dprob = do @ v.t()
                dscore = prob * (dprob - (prob * dprob).sum(1, keepdim=True)) * s["scale"]
                res["dq"][a:b, col] = dscore @ k
                res["dk"][a:b, kcol] += dscore.t() @ q
                res["dv"][a:b, kcol] += prob.t() @ do
    return res


def _exact_cached(s):
    h, hkv, d, b, p, g = s["heads"], s["kv_heads"], s["dim"], s["block"], s["prefix"], s["heads"] // s["kv_heads"]
    lens = s["suffix_len"].tolist()
    out = torch.zeros(len(lens) * b, h * d, dtype=torch.float64, device=DEV)
    shared = [x[s["prefix_pages"].long()].reshape(-1, hkv, d)[:p].double() for x in (s["k_pages"], s["v_pages"])]
    for i, length in enumerate(lens):
        mine = [x[s["page_table"][i].long()].reshape(-1, hkv, d)[:length].double() for x in (s["k_pages"], s["v_pages"])]
        k, v = (torch.cat([x, y]).permute(1, 0, 2).contiguous() for x, y in zip(shared, mine))
        q = s["q"][i * b:(i + 1) * b].double().reshape(b, hkv, g, d).permute(1, 0, 2, 3).reshape(hkv, b * g, d)
        score = (torch.matmul(q, k.transpose(1, 2)) * s["scale"]).reshape(hkv, b, g, p + length)
        seen = p + length - b + torch.arange(b, device=DEV)
        score = score.masked_fill((torch.arange(p + length, device=DEV) > seen[:, None])[None, :, None, :], -math.inf)
        prob = _softmax64(score)[0].reshape(hkv, b * g, p + length)
        out[i * b:(i + 1) * b] = torch.matmul(prob, v).reshape(hkv, b, g, d).permute(1, 0, 2, 3).reshape(b, h * d)
    return {"out": out}
