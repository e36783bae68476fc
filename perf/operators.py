"""Workloads of the transformer-layer operators: RMS norm, expert routing, prompt attention and paged decode attention.

Each case is one call as a serving program makes it around the tensor- and expert-parallel products of this library.
``run`` computes it in plain torch operations in 32 bits, or, where ``own`` is true, through the library's entry points;
``exact`` computes it once more in 64 bits from the definition.

The definitions:

* norm    s = x + residual;  y = s / sqrt(mean(s^2) + eps) * weight, over rows of ``width``.  Outputs s (the new residual)
          and y.  An 8-bit y is e4m3(y / scale), with scale = max(max|y| / 448, 2^-126) over the row or over each block of
          128 columns.
* gate    score = softmax(logits) or sigmoid(logits).  The top-k experts are chosen by score + bias (without a bias by the
          logit itself, which orders them alike), largest first, equal ones by the lower id; with groups, only among the
          experts of the best groups (by the sum of each group's two largest choice values).  gate = the chosen scores,
          divided by their sum if asked for, times ``scale``.
* prompt  packed sequences: softmax(q k^T / sqrt(d) + mask) v.  Query i of a sequence of Lq queries and Lk keys sees keys
          0 .. i + Lk - Lq.  Query head h reads key head h / (hq / hkv).  Also the log of the softmax's sum (lse).
* decode  the same for one new token of each sequence, whose keys and values lie in the pages of a cache.
"""
import functools
import math
import random

import torch

own = False

DEVICE = "cuda:0"
EPS = 1e-6
F8_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "f8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "f8": 1}


def listed():
    return [
        # one token through a layer of width 8192: a decode step's norm, where only the call's latency counts
        dict(name="norm_token", op="norm", rows=1, width=8192, x="bf16", out="bf16", block=0),
        # a rank's rows of a 16384 x 8192 activation, fp32 as GEMM + ReduceScatter leaves them, normed for the next AllGather
        dict(name="norm_rank_rows", op="norm", rows=2048, width=8192, x="f32", out="bf16", block=0),
        # a whole batch of odd size at width 5120, in 8 bits with a scale for each 128 columns, for an AllGather of half the bytes
        dict(name="norm_8bit", op="norm", rows=8191, width=5120, x="bf16", out="f8", block=128),
        # the router of a decode step: 16 tokens, 64 experts
        dict(name="gate_tokens", op="gate", rows=16, experts=64, topk=8, score="softmax", bias=False, groups=1, keep=1,
             renorm=True, scale=1.0, x="f32"),
        # the router of the 4096-token MoE layer
        dict(name="gate_layer", op="gate", rows=4096, experts=64, topk=8, score="softmax", bias=False, groups=1, keep=1,
             renorm=True, scale=1.0, x="f32"),
        # a large prompt batch of odd size, 256 experts in 8 groups, sigmoid scores with a balance bias
        dict(name="gate_groups", op="gate", rows=16381, experts=256, topk=8, score="sigmoid", bias=True, groups=8, keep=4,
             renorm=True, scale=2.5, x="f32"),
        # short prompts of different lengths packed into one batch, a rank's eight query heads and one key head
        dict(name="prompt_packed", op="prompt", seqs=16, longest=1500, shortest=1, prefix=0, hq=8, hkv=1, d=128, lens=3),
        # one prompt of 16384 tokens
        dict(name="prompt_long", op="prompt", seqs=1, longest=16384, shortest=16384, prefix=0, hq=8, hkv=1, d=128, lens=1),
        # the last pieces of prompts whose first 6000 tokens have been computed before, narrow heads
        dict(name="prompt_pieces", op="prompt", seqs=3, longest=700, shortest=300, prefix=6000, hq=16, hkv=4, d=64, lens=5),
        # one user's next token over a short cache
        dict(name="decode_one", op="decode", seqs=1, longest=777, shortest=777, hq=8, hkv=1, d=128, page=16, order="slot", lens=1),
        # a batch of users with caches of all lengths and a few idle slots
        dict(name="decode_batch", op="decode", seqs=128, longest=16000, shortest=1, hq=8, hkv=1, d=128, page=16, order="slot", lens=2),
        # a few users with very long caches, all heads on one GPU, pages kept head by head
        dict(name="decode_long", op="decode", seqs=4, longest=131072, shortest=90000, hq=64, hkv=8, d=128, page=64, order="head", lens=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gate", "prompt", "decode"])
    if op == "norm":
        width = rng.choice([2048, 5120, 8192, _log(rng, 64, 8192), 8 * _log(rng, 8, 1024)])
        return dict(op=op, rows=_log(rng, 1, min(8191, 2 ** 22 * 6 // width)), width=width, x=rng.choice(["bf16", "f32"]),
                    out=rng.choice(["bf16", "f8"]), block=rng.choice([0, 128]))
    if op == "gate":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * _log(rng, 8, 256 // groups)
        keep = rng.randint((groups + 1) // 2, groups)
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, rows=_log(rng, 1, 16381), experts=experts, topk=rng.choice([1, 2, 4, 6, 8]), score=score,
                    bias=score == "sigmoid" or groups > 1, groups=groups, keep=keep, renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), x=rng.choice(["f32", "bf16"]))
    hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 5, 8])
    if op == "prompt":
        hkv = min(hkv, 4)
        longest, prefix = _log(rng, 1, 8192), rng.choice([0, 0, _log(rng, 1, 4096)])
        while hkv * group * longest * (longest + prefix) > 16384 * 8192 * 8:
            longest = longest * 2 // 3
        most = 16384 * 8192 * 8 // (hkv * group * longest * (longest + prefix))
        return dict(op=op, seqs=rng.randint(1, min(24, most)), longest=longest, shortest=rng.randint(1, longest), prefix=prefix,
                    hq=hkv * group, hkv=hkv, d=rng.choice([64, 128]), lens=rng.randrange(10 ** 6))
    longest = _log(rng, 1, 65536)
    most = max(1, min(256, 4 * 90000 * 8 // (2 * longest * hkv)))
    return dict(op=op, seqs=rng.randint(1, most), longest=longest, shortest=rng.randint(1, longest), hq=hkv * group, hkv=hkv,
                d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), order=rng.choice(["slot", "head"]),
                lens=rng.randrange(10 ** 6))


def lengths(case):
    """Lengths of the case's sequences: spread over their logarithm, one of them the longest; a decode batch of eight or
    more holds some idle slots of length 0."""
    r = random.Random(case["lens"])
    n = [case["longest"]] + [_log(r, case["shortest"], case["longest"]) for _ in range(case["seqs"] - 1)]
    if case["op"] == "decode" and len(n) >= 8:
        for i in r.sample(range(1, len(n)), len(n) // 16 + 1):
            n[i] = 0
    r.shuffle(n)
    return n


def work(case):
    if case["op"] == "norm":
        n, w = case["rows"] * case["width"], case["width"]
        scales = case["rows"] * (-(-w // case["block"]) if case["block"] else 1) * 4 if case["out"] == "f8" else 0
        return {"bytes": n * (BYTES[case["x"]] + 2 + 2 + BYTES[case["out"]]) + 2 * w + scales, "flops": 5 * n}
    if case["op"] == "gate":
        n = case["rows"] * case["experts"]
        return {"bytes": n * BYTES[case["x"]] + case["rows"] * case["topk"] * 8 + 4 * case["experts"] * case["bias"], "flops": 5 * n}
    n, d = lengths(case), case["d"]
    if case["op"] == "prompt":
        pairs = sum(q * case["prefix"] + q * (q + 1) // 2 for q in n)
        tokens, keys = sum(n), sum(n) + case["prefix"] * len(n)
        return {"bytes": 2 * d * (2 * tokens * case["hq"] + 2 * keys * case["hkv"]) + 4 * tokens * case["hq"],
                "flops": 4 * d * case["hq"] * pairs}
    pages = sum(-(-x // case["page"]) for x in n)
    return {"bytes": 4 * d * case["hkv"] * sum(n) + len(n) * case["hq"] * (4 * d + 4) + 4 * pages,
            "flops": 4 * d * case["hq"] * sum(n)}


# ---------------------------------------------------------------- inputs

def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32) * std).to(dtype)


def _gate_inputs(case, g):
    """Logits as a router gives them: an offset for each expert (so the experts' loads differ) and a spread of 1.5.  A token
    whose choice would hang on a difference of rounding size is drawn again, so that every way to round chooses alike."""
    rows, experts = case["rows"], case["experts"]
    offset = torch.randn(experts, generator=g, device=DEVICE) * 0.5
    bias = torch.randn(experts, generator=g, device=DEVICE) * 0.05 if case["bias"] else None
    logits = torch.empty(rows, experts, device=DEVICE, dtype=TYPES[case["x"]])
    todo = torch.arange(rows, device=DEVICE)
    for _ in range(50):
        new = torch.randn(len(todo), experts, generator=g, device=DEVICE) * 1.5 + offset
        logits[todo] = new.to(logits.dtype)
        if bias is None:
            break  # chosen by the logits themselves: nothing is rounded, and equal ones go by their ids
        at = logits[todo].double()
        c = (at.softmax(1) if case["score"] == "softmax" else at.sigmoid()) + bias.double()
        near = torch.zeros(len(todo), device=DEVICE, dtype=torch.bool)
        if case["groups"] > 1:
            by = c.view(len(todo), case["groups"], -1).topk(2, dim=2).values.sum(2).sort(1, descending=True)
            near = (by.values.diff(dim=1).abs() < 2e-6).any(1)
            kept = torch.zeros(len(todo), case["groups"], device=DEVICE, dtype=torch.bool)
            kept.scatter_(1, by.indices[:, :case["keep"]], True)
            c = c.masked_fill(~kept.repeat_interleave(experts // case["groups"], 1), -math.inf)
        near |= (c.sort(1, descending=True).values[:, :case["topk"] + 1].diff(dim=1).abs() < 1e-6).any(1)
        todo = todo[near]
        if not len(todo):
            break
    return logits, bias


def _cu(n):
    return torch.tensor([0] + n, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEVICE)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        rows, width = case["rows"], case["width"]
        s["x"] = _normal(g, (rows, width), TYPES[case["x"]], 0.3)
        s["residual"] = _normal(g, (rows, width), torch.bfloat16)
        s["weight"] = (1.0 + 0.1 * torch.randn(width, generator=g, device=DEVICE)).to(torch.bfloat16)
        s["sum"] = torch.empty_like(s["residual"])
        s["out"] = torch.empty(rows, width, device=DEVICE, dtype=TYPES[case["out"]])
        s["scales"] = None
        if case["out"] == "f8":
            s["scales"] = torch.empty(rows, -(-width // case["block"]) if case["block"] else 1, device=DEVICE)
        return s
    if case["op"] == "gate":
        s["logits"], s["bias"] = _gate_inputs(case, g)
        s["ids"] = torch.empty(case["rows"], case["topk"], device=DEVICE, dtype=torch.int32)
        s["gate"] = torch.empty(case["rows"], case["topk"], device=DEVICE)
        return s
    n, hq, hkv, d = lengths(case), case["hq"], case["hkv"], case["d"]
    if case["op"] == "prompt":
        tokens = sum(n)
        s["n"] = n
        s["cu_q"] = _cu(n)
        if case["prefix"]:
            s["q"] = _normal(g, (tokens, hq, d), torch.bfloat16)
            keys = tokens + case["prefix"] * len(n)
            s["k"], s["v"] = (_normal(g, (keys, hkv, d), torch.bfloat16) for _ in range(2))
            s["cu_k"] = _cu([x + case["prefix"] for x in n])
        else:  # one product gives queries, keys and values side by side
            qkv = _normal(g, (tokens, hq + 2 * hkv, d), torch.bfloat16)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
            s["cu_k"] = s["cu_q"]
        s["out"] = torch.empty(tokens, hq, d, device=DEVICE, dtype=torch.bfloat16)
        s["lse"] = torch.empty(tokens, hq, device=DEVICE)
        return s
    page = case["page"]
    count = [-(-x // page) for x in n]
    pages = sum(count) + 3
    shape = (pages, page, hkv, d) if case["order"] == "slot" else (pages, hkv, page, d)
    s["k"], s["v"] = (_normal(g, shape, torch.bfloat16) for _ in range(2))
    if case["order"] == "head":
        s["k"], s["v"] = s["k"].transpose(1, 2), s["v"].transpose(1, 2)
    s["q"] = _normal(g, (len(n), hq, d), torch.bfloat16, 1.5)
    # the pages of a sequence lie anywhere in the cache
    anywhere = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    first = torch.tensor([0] + count).cumsum(0)[:-1].to(DEVICE)
    at = first[:, None] + torch.arange(max(count), device=DEVICE)
    s["table"] = anywhere[at.clamp(max=pages - 1)].contiguous()
    s["lens"] = torch.tensor(n, dtype=torch.int32, device=DEVICE)
    s["out"] = torch.empty(len(n), hq, d, device=DEVICE, dtype=torch.bfloat16)
    s["lse"] = torch.empty(len(n), hq, device=DEVICE)
    return s


# ---------------------------------------------------------------- the plain forms

def _norm(s):
    case = s["case"]
    total = s["x"].float() + s["residual"].float()
    y = total * torch.rsqrt(total.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    if case["out"] != "f8":
        return {"sum": total.to(torch.bfloat16), "out": y.to(TYPES[case["out"]])}
    rows, width = y.shape
    block = case["block"] or width
    wide = torch.nn.functional.pad(y, (0, -width % block)).view(rows, -1, block)
    scales = (wide.abs().amax(2) / F8_MAX).clamp(min=2.0 ** -126)
    q = (wide / scales[:, :, None]).view(rows, -1)[:, :width].clamp(-F8_MAX, F8_MAX)
    return {"sum": total.to(torch.bfloat16), "out": q.to(TYPES["f8"]), "scales": scales}


def _gate(s):
    case = s["case"]
    x = s["logits"].float()
    score = x.softmax(1) if case["score"] == "softmax" else x.sigmoid()
    choice = x if s["bias"] is None else score + s["bias"]
    if case["groups"] > 1:
        by = choice.view(len(x), case["groups"], -1).topk(2, dim=2).values.sum(2)
        kept = torch.zeros_like(by, dtype=torch.bool)
        kept.scatter_(1, by.sort(dim=1, descending=True, stable=True).indices[:, :case["keep"]], True)
        choice = choice.masked_fill(~kept.repeat_interleave(x.shape[1] // case["groups"], 1), -math.inf)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :case["topk"]]
    gate = score.gather(1, ids)
    if case["renorm"]:
        gate = gate / gate.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "gate": gate * case["scale"]}


def _attention(q, k, v, mask):
    """q: n x hq x lq x d, k and v: n x hkv x lk x d, mask (seen keys): n x lq x lk; all in 32 bits."""
    n, hq, lq, d = q.shape
    hkv, lk = k.shape[1], k.shape[2]
    score = (q.reshape(n * hkv, -1, d) @ k.reshape(n * hkv, lk, d).transpose(1, 2)).view(n, hq, lq, lk) / math.sqrt(d)
    score = score.masked_fill_(~mask[:, None], -math.inf)
    top = score.amax(3, keepdim=True)
    weight = score.sub_(top.clamp(min=-1e30)).exp_()
    total = weight.sum(3, keepdim=True)
    out = (weight.view(n * hkv, -1, lk) @ v.reshape(n * hkv, lk, d)).view(n, hq, lq, d)
    out = torch.where(total > 0, out / total, 0.0)
    return out, (top + total.log()).squeeze(3)


def _spread(x, cu, longest):
    """The packed rows as n x heads x longest x d in 32 bits, and which places hold a row."""
    n = cu[1:] - cu[:-1]
    at = torch.arange(longest, device=x.device)
    held = at < n[:, None]
    rows = (cu[:-1, None] + at).clamp(max=max(x.shape[0] - 1, 0)).long()
    return torch.where(held[:, :, None, None], x[rows].float(), 0.0).transpose(1, 2), held


def _prompt(s):
    case = s["case"]
    longest = max(s["n"])
    q, held_q = _spread(s["q"], s["cu_q"], longest)
    k, held_k = _spread(s["k"], s["cu_k"], longest + case["prefix"])
    v, _ = _spread(s["v"], s["cu_k"], longest + case["prefix"])
    i, j = torch.arange(q.shape[2], device=DEVICE), torch.arange(k.shape[2], device=DEVICE)
    mask = (j <= i[:, None] + case["prefix"]) & held_k[:, None, :]
    out, lse = _attention(q, k, v, mask)
    return {"out": out.transpose(1, 2)[held_q].to(torch.bfloat16), "lse": lse.transpose(1, 2)[held_q]}


def _decode(s):
    table, lens, page = s["table"], s["lens"], s["case"]["page"]
    hkv, d = s["case"]["hkv"], s["case"]["d"]
    mask = torch.arange(table.shape[1] * page, device=DEVICE) < lens[:, None]
    k, v = (s[x][table.long()].reshape(len(lens), -1, hkv, d).float().transpose(1, 2) for x in "kv")
    out, lse = _attention(s["q"].float()[:, :, None], k, v, mask[:, None])
    return {"out": out[:, :, 0].to(torch.bfloat16), "lse": lse[:, :, 0]}


# ---------------------------------------------------------------- one pass

@functools.lru_cache(None)
def _sgt():
    import signal_gated_tiled_amd
    return signal_gated_tiled_amd


def _run_own(s):
    sgt, case = _sgt(), s["case"]
    if case["op"] == "norm":
        sgt.rms_norm(s["x"], s["weight"], s["out"], residual=s["residual"], sum_out=s["sum"], scales=s["scales"], eps=EPS)
        got = {"sum": s["sum"], "out": s["out"]}
        if s["scales"] is not None:
            got["scales"] = s["scales"]
        return got
    if case["op"] == "gate":
        sgt.moe_gate(s["logits"], s["ids"], s["gate"], bias=s["bias"], score=case["score"], n_group=case["groups"],
                     topk_group=case["keep"], group_top=2, renormalize=case["renorm"], scale=case["scale"])
        return {"ids": s["ids"], "gate": s["gate"]}
    if case["op"] == "prompt":
        sgt.attn_prompt(s["q"], s["k"], s["v"], s["out"], s["cu_q"], s["cu_k"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if "workspace" not in s:  # a serving program keeps one for its batches
        s["workspace"] = torch.zeros(sgt.attn_decode_workspace(len(s["lens"]), case["hq"], case["hkv"], case["d"]),
                                     dtype=torch.uint8, device=DEVICE)
    sgt.attn_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["out"], s["workspace"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm, "gate": _gate, "prompt": _prompt, "decode": _decode}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_rows(q, k, v, seen):
    """One sequence: q lq x hq x d, k and v lk x hkv x d; seen[i]: how many keys, from the first, query i sees."""
    lq, hq, d = q.shape
    lk, hkv = k.shape[0], k.shape[1]
    out = torch.zeros(lq, hq, d, device=q.device, dtype=torch.float64)
    lse = torch.full((lq, hq), -math.inf, device=q.device, dtype=torch.float64)
    for h in range(hq):
        kh, vh = k[:, h * hkv // hq].double(), v[:, h * hkv // hq].double()
        for a in range(0, lq, 4096):
            here = seen[a:a + 4096]
            if lk == 0:
                continue
            z = torch.mm(q[a:a + 4096, h].double(), kh.t()) * d ** -0.5
            z[torch.arange(lk, device=q.device)[None, :] >= here[:, None]] = -math.inf
            lse[a:a + 4096, h] = torch.logsumexp(z, 1)
            some = here > 0
            p = torch.exp(z[some] - lse[a:a + 4096, h][some][:, None])
            out[a:a + 4096, h][some] = torch.mm(p, vh)
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        t = s["x"].double() + s["residual"].double()
        y = t / (t.pow(2).sum(1, keepdim=True) / case["width"] + EPS).sqrt() * s["weight"].double()
        got = {"sum": t, "out": y}
        if case["out"] == "f8":
            block = case["block"] or case["width"]
            scales = [y[:, a:a + block].abs().max(1).values / F8_MAX for a in range(0, case["width"], block)]
            got["scales"] = torch.stack(scales, 1)
            got["out"] = torch.cat([y[:, j * block:(j + 1) * block] / x[:, None] for j, x in enumerate(scales)], 1)
        return got
    if case["op"] == "gate":
        x = s["logits"].double()
        e = torch.exp(x - x.max(1, keepdim=True).values)
        score = e / e.sum(1, keepdim=True) if case["score"] == "softmax" else 1 / (1 + torch.exp(-x))
        choice = x.clone() if s["bias"] is None else score + s["bias"].double()
        if case["groups"] > 1:
            parts = choice.split(case["experts"] // case["groups"], 1)
            best = torch.stack([p.sort(1, descending=True).values[:, :2].sum(1) for p in parts], 1)
            for _ in range(case["groups"] - case["keep"]):  # the worst group goes, of equal ones the last
                low = best == best.amin(1, keepdim=True)
                worst = case["groups"] - 1 - low.flip(1).long().argmax(1)
                best.scatter_(1, worst[:, None], math.inf)
                gone = worst[:, None] == torch.arange(case["experts"], device=DEVICE)[None] // len(parts[0][0])
                choice[gone] = -math.inf
        ids, gate = [], []
        for _ in range(case["topk"]):  # one expert after another, of equal ones the first
            i = (choice == choice.amax(1, keepdim=True)).long().argmax(1, keepdim=True)
            ids.append(i)
            gate.append(score.gather(1, i))
            choice.scatter_(1, i, -math.inf)
        gate = torch.cat(gate, 1)
        if case["renorm"]:
            gate = gate / gate.sum(1, keepdim=True)
        return {"ids": torch.cat(ids, 1).to(torch.int32), "gate": gate * case["scale"]}
    parts = []
    if case["op"] == "prompt":
        a = b = 0
        for n in s["n"]:
            m = n + case["prefix"]
            seen = torch.arange(n, device=DEVICE) + 1 + case["prefix"]
            parts.append(_exact_rows(s["q"][a:a + n], s["k"][b:b + m], s["v"][b:b + m], seen))
            a, b = a + n, b + m
        return {"out": torch.cat([p[0] for p in parts]), "lse": torch.cat([p[1] for p in parts])}
    for b, n in enumerate(lengths(case)):
        j = torch.arange(n, device=DEVICE)
        page, slot = s["table"][b].long()[j // case["page"]], j % case["page"]
        parts.append(_exact_rows(s["q"][b:b + 1], s["k"][page, slot], s["v"][page, slot], torch.tensor([n], device=DEVICE)))
    return {"out": torch.cat([p[0] for p in parts]), "lse": torch.cat([p[1] for p in parts])}
