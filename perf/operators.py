"""Cases of the paged-batch operators (append, attention with a shared prefix, attention
weights, eviction by accumulated weight): inputs, the operators' plain forms in elementary
torch operations, and their definition in 64 bits.

Layouts. K and V live in pools [pages][kv heads][page size][head dim]; sequence b holds its
tokens in the slots of its row of the page table, in order, `lengths[b]` of them. Queries
and new keys are ragged rows: sequence b's are [row_start[b], row_start[b + 1]).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------------------- the cases

def _attend(name, **kw):
    c = dict(op="attend", dtype="bf16", b=4, n=1, ragged_rows=False, hq=16, hkv=16, d=64, page=16, prefix=0,
             length=256, causal=False)
    c.update(kw)
    return dict(name=name, **c) if name else c


def _weights(name, **kw):
    c = dict(op="weights", dtype="bf16", b=4, n=1, ragged_rows=False, hq=16, hkv=16, d=64, page=16, length=256,
             causal=False)
    c.update(kw)
    return dict(name=name, **c) if name else c


def _append(name, **kw):
    c = dict(op="append", dtype="bf16", b=4, n=1, ragged_rows=False, hkv=16, d=64, page=16, length=256)
    c.update(kw)
    return dict(name=name, **c) if name else c


def _evict(name, **kw):
    # n: tokens appended before each eviction (a steady state at `keep` tokens); 0: one
    # eviction from `length` tokens down to `keep`
    c = dict(op="evict", dtype="bf16", b=4, n=1, hkv=16, d=64, page=16, length=0, keep=256, sinks=4, recent=64)
    c.update(kw)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # four streams at their first frames, one query token each: the call's own latency
        _attend("attend_small", b=4, n=1, hq=16, hkv=16, prefix=500, length=107, causal=True),
        # a server's decode step: 64 answers behind one long instruction
        _attend("attend_decode", b=64, n=1, hq=32, hkv=8, d=128, prefix=16384, length=1024, causal=True),
        # two camera streams localised against the same 8 scale frames, 8 frames of their own
        _attend("attend_frames", b=2, n=1004, hq=16, hkv=16, prefix=8032, length=8032, causal=False),
        # drafted tokens checked in fp32, rows of unequal length
        _attend("attend_drafts_f32", dtype="f32", b=8, n=5, ragged_rows=True, hq=16, hkv=4, prefix=1500, length=700,
                causal=True),
        # the weights of one decode step, per cached token
        _weights("weights_decode", b=32, n=1, hq=32, hkv=8, d=128, length=8192, causal=True),
        # a frame's 1,004 queries over 16 cached frames
        _weights("weights_frame", b=1, n=1004, hq=16, hkv=16, length=16064, causal=False),
        # a short fp32 step with drafts
        _weights("weights_drafts_f32", dtype="f32", b=6, n=4, ragged_rows=True, hq=16, hkv=4, length=600, causal=True),
        # drafts appended again after a verifier took the last ones back
        _append("append_drafts", b=64, n=5, ragged_rows=True, hkv=8, d=128, length=4096),
        # two streams' frames
        _append("append_frames", b=2, n=1004, hkv=16, length=8032),
        # one token in, one token out
        _evict("evict_step", b=64, n=1, hkv=8, d=128, keep=4096, sinks=4, recent=512),
        # a frame in, as many tokens out, fp32
        _evict("evict_frame_f32", dtype="f32", b=2, n=1004, hkv=16, d=64, keep=8192, sinks=5, recent=2008),
        # after a long prompt: 32k tokens down to 4k
        _evict("evict_prompt", b=4, n=0, hkv=8, d=128, length=32768, keep=4096, sinks=4, recent=512),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def heads(c):
        c["hkv"] = rng.choice([1, 2, 3, 4, 8, 16])
        g = rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
        if "hq" in c:
            c["hq"] = c["hkv"] * g
        c["d"] = rng.choice([64, 128])
        c["page"] = rng.choice([16, 16, 32, 64])
        c["dtype"] = rng.choice(["bf16", "bf16", "bf16", "f32"])
        return g

    while True:
        op = rng.choice(["attend", "attend", "weights", "weights", "append", "evict", "evict"])
        if op == "attend":
            c = _attend(None)
            g = heads(c)
            c["b"], c["n"] = log(1, 128), rng.choice([1, 1, rng.randint(2, 8), log(9, 1200)])
            c["prefix"] = rng.choice([0, log(1, 32768), log(64, 32768)])
            c["length"], c["causal"] = log(1, 16384), rng.random() < 0.6
            c["ragged_rows"] = rng.random() < 0.5
            rows, keys = c["b"] * c["n"] * c["hkv"] * g, c["prefix"] + c["length"]
            size = rows * keys                                   # logits of the plain form
            held = (c["b"] * c["length"] + c["prefix"]) * c["hkv"] * c["d"]
            if c["n"] > c["length"] or size > 5.1e8 or held > 1.3e8 or (c["dtype"] == "f32" and size > 1.2e8):
                continue
        elif op == "weights":
            c = _weights(None)
            g = heads(c)
            c["b"], c["n"] = log(1, 64), rng.choice([1, 1, rng.randint(2, 8), log(9, 1200)])
            c["length"], c["causal"] = log(1, 32768), rng.random() < 0.6
            c["ragged_rows"] = rng.random() < 0.5
            size = c["b"] * c["n"] * c["hkv"] * g * c["length"]
            if c["n"] > c["length"] or size > 2.5e8 or c["b"] * c["length"] * c["hkv"] * c["d"] > 2.6e8 or (
                    c["dtype"] == "f32" and size > 6e7):
                continue
        elif op == "append":
            c = _append(None)
            heads(c)
            c["b"], c["n"], c["length"] = log(1, 128), log(1, 2048), log(1, 16384)
            c["ragged_rows"] = rng.random() < 0.5
            if c["b"] * (c["length"] + c["n"]) * c["hkv"] * c["d"] > 2.6e8 or c["b"] * c["n"] > 16384:
                continue
        else:
            c = _evict(None)
            heads(c)
            c["b"], c["keep"] = log(1, 128), log(8, 16384)
            c["sinks"] = rng.randint(0, min(8, c["keep"] // 4))
            c["recent"] = rng.randint(0, c["keep"] // 2)
            if rng.random() < 0.5:
                c["n"], c["length"] = log(1, 1200), 0
            else:
                c["n"], c["length"] = 0, c["keep"] + log(1, 16384)
            if c["b"] * (c["length"] + c["n"] + c["keep"]) * c["hkv"] * c["d"] > 2.6e8:
                continue
        return c


# ---------------------------------------------------------------------------- inputs

def _spread(b, most, ragged):
    """b whole numbers up to `most`, the same ones for every seed: half to all of it."""
    if not ragged or b == 1:
        return [most] * b
    lo = max(1, most // 2)
    return [lo + (most - lo) * i // (b - 1) for i in range(b)]


def _lengths(c):
    if c["op"] == "evict":
        if c["n"]:
            return [c["keep"]] * c["b"]
        lo = c["keep"] + (c["length"] - c["keep"]) // 2
        return [c["length"] - (c["length"] - lo) * i // max(1, c["b"] - 1) for i in range(c["b"])]
    return [max(x, c["n"]) for x in _spread(c["b"], c["length"], True)]


def _rows(c):
    return _spread(c["b"], c["n"], c.get("ragged_rows", False))


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    dt = DTYPES[c["dtype"]]
    b, hkv, d, page = c["b"], c["hkv"], c["d"], c["page"]
    perm = torch.randperm(b, generator=g, device=DEV)
    lengths = torch.tensor(_lengths(c), dtype=torch.int32).to(DEV)[perm].contiguous()
    rows = torch.tensor(_rows(c), dtype=torch.int32).to(DEV)[torch.randperm(b, generator=g, device=DEV)]
    row_start = torch.zeros(b + 1, dtype=torch.int32, device=DEV)
    row_start[1:] = torch.cumsum(rows, 0)
    total = sum(_rows(c))
    room = max(_lengths(c)) + (c["n"] if c["op"] in ("append", "evict") else 0)
    max_pages = -(-room // page)
    prefix = c.get("prefix", 0)
    pp = -(-prefix // page)
    pages = b * max_pages + pp
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    s = dict(c=c, lengths=lengths, row_start=row_start, max_rows=max(_rows(c)),
             prefix_pages=order[:pp].contiguous(), page_table=order[pp:].view(b, max_pages).contiguous(), own=None)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(dt)

    # values with a mean per channel, as trained models have them
    s["k_pool"] = normal(pages, hkv, page, d)
    s["v_pool"] = normal(pages, hkv, page, d).add_(normal(1, hkv, 1, d, scale=0.3))
    if c["op"] in ("attend", "weights"):
        s["scale"] = 1.0 / math.sqrt(d)
        s["q"] = normal(total, c["hq"], d, scale=2.0)
    if c["op"] == "attend":
        s["o"] = torch.zeros(total, c["hq"], d, device=DEV, dtype=dt)
        s["lse"] = torch.zeros(total, c["hq"], device=DEV)
    if c["op"] == "weights":
        s["lse"] = _logits_lse(s)
        s["scores"] = torch.rand(b, hkv, max_pages * page, generator=g, device=DEV)
    if c["op"] in ("append", "evict"):
        s["k"], s["v"] = normal(total, hkv, d), normal(total, hkv, d)
        s["scores"] = torch.exp(2.0 * torch.randn(b, hkv, max_pages * page, generator=g, device=DEV))
        # positions of the cached tokens, oldest first, some gone already
        gone = torch.randint(0, 1 + max(1, room // 4), (b, 1, 1), generator=g, device=DEV)
        at = torch.arange(max_pages * page, device=DEV).view(1, 1, -1)
        s["positions"] = torch.where(at < c.get("sinks", 0), at, at + gone).expand(b, hkv, -1).to(
            torch.int32).contiguous()
        s["next_positions"] = (lengths + gone.view(-1)).to(torch.int32)
        s["lengths0"], s["next0"] = lengths.clone(), s["next_positions"].clone()
        if c["op"] == "evict" and not c["n"]:
            s["scores0"], s["positions0"] = s["scores"].clone(), s["positions"].clone()
    return s


# ---------------------------------------------------------------------------- plain forms

def _private(s, pool):
    """[B, kv heads, slots, d] of the sequences' own pages, in fp32."""
    t = pool[s["page_table"].long()]
    b, p, h, e, d = t.shape
    return t.permute(0, 2, 1, 3, 4).reshape(b, h, p * e, d).float()


def _prefix(s, pool):
    t = pool[s["prefix_pages"].long()]
    p, h, e, d = t.shape
    return t.permute(1, 0, 2, 3).reshape(h, p * e, d)[:, : s["c"]["prefix"]].float()


def _padded_rows(s):
    """Row numbers [B, n] of the ragged rows and which of them are there."""
    at = torch.arange(s["max_rows"], device=DEV).view(1, -1)
    there = at < (s["row_start"][1:] - s["row_start"][:-1]).view(-1, 1)
    rows = torch.where(there, s["row_start"][:-1].view(-1, 1) + at, torch.zeros_like(at))
    return rows.long(), there


def _queries(s, rows):
    """[B, kv heads, n * group, d] in fp32, scaled."""
    c = s["c"]
    g = c["hq"] // c["hkv"]
    q = s["q"][rows].float() * s["scale"]
    b, n = rows.shape
    return q.view(b, n, c["hkv"], g, c["d"]).permute(0, 2, 1, 3, 4).reshape(b, c["hkv"], n * g, c["d"])


def _hidden(s, slots):
    """[B, 1, n * group, slots]: keys that a row does not see."""
    c = s["c"]
    g = c["hq"] // c["hkv"]
    n = s["max_rows"]
    limit = s["lengths"].view(-1, 1).expand(-1, n)
    if c["causal"]:
        count = (s["row_start"][1:] - s["row_start"][:-1]).view(-1, 1)
        limit = torch.minimum(limit, limit - count + torch.arange(n, device=DEV).view(1, -1) + 1)
    limit = limit.repeat_interleave(g, 1)
    return torch.arange(slots, device=DEV).view(1, 1, 1, -1) >= limit.view(c["b"], 1, n * g, 1)


def _private_logits(s):
    rows, there = _padded_rows(s)
    q = _queries(s, rows)
    k = _private(s, s["k_pool"])
    x = q @ k.transpose(2, 3)
    return x.masked_fill_(_hidden(s, k.shape[2]), -math.inf), q, rows, there


def _per_row(s, x, rows, there, out):
    """Values [B, kv heads, n * group, ...] written to the rows of out [rows, heads, ...]."""
    c = s["c"]
    g = c["hq"] // c["hkv"]
    b, n = rows.shape
    x = x.view(b, c["hkv"], n, g, *x.shape[3:]).transpose(1, 2).reshape(b, n, c["hq"], *x.shape[3:])
    out[rows[there]] = x[there].to(out.dtype)
    return out


def _logits_lse(s):
    x, _, rows, there = _private_logits(s)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    lse = torch.log(torch.exp(x - m).sum(-1)) + m[..., 0]
    return _per_row(s, lse, rows, there, torch.zeros(s["q"].shape[:2], device=DEV))


def _plain_attend(s):
    c = s["c"]
    x, q, rows, there = _private_logits(s)
    b, h, r, _ = q.shape
    m = x.amax(-1, keepdim=True)
    if c["prefix"]:
        kp = _prefix(s, s["k_pool"])
        y = q.transpose(0, 1).reshape(h, b * r, c["d"]) @ kp.transpose(1, 2)
        m = torch.maximum(m, y.amax(-1).view(h, b, r, 1).transpose(0, 1))
    m = m.clamp_min(-1e30)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = x @ _private(s, s["v_pool"])
    if c["prefix"]:
        y = y.sub_(m.transpose(0, 1).reshape(h, b * r, 1)).exp_()
        total = total + y.sum(-1).view(h, b, r, 1).transpose(0, 1)
        o = o + (y @ _prefix(s, s["v_pool"])).view(h, b, r, c["d"]).transpose(0, 1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = torch.where(total > 0, torch.log(total) + m, torch.full_like(m, -math.inf))
    return {"o": _per_row(s, o, rows, there, s["o"]), "lse": _per_row(s, lse[..., 0], rows, there, s["lse"])}


def _plain_weights(s):
    c = s["c"]
    x, _, rows, there = _private_logits(s)
    b, n = rows.shape
    g = c["hq"] // c["hkv"]
    lse = torch.where(there.unsqueeze(-1), s["lse"][rows], torch.full_like(s["lse"][rows], math.inf))
    lse = lse.view(b, n, c["hkv"], g).permute(0, 2, 1, 3).reshape(b, c["hkv"], n * g, 1)
    s["scores"] += x.sub_(lse).exp_().sum(2)
    return {"scores": s["scores"]}


def _plain_append(s):
    page = s["c"]["page"]
    rows, there = _padded_rows(s)
    at = s["lengths"].long().view(-1, 1) + torch.arange(s["max_rows"], device=DEV).view(1, -1)
    b_of = torch.arange(s["c"]["b"], device=DEV).view(-1, 1).expand_as(at)[there]
    at, rows = at[there], rows[there]
    phys = s["page_table"][b_of, at // page].long()
    # a page that is begun is cleared first
    fresh = at % page == 0
    s["k_pool"][phys[fresh]] = 0
    s["v_pool"][phys[fresh]] = 0
    s["k_pool"][phys, :, at % page] = s["k"][rows]
    s["v_pool"][phys, :, at % page] = s["v"][rows]
    s["scores"][b_of, :, at] = 0
    first = (s["next_positions"] - s["lengths"]).long()
    s["positions"][b_of, :, at] = (first[b_of] + at).to(torch.int32).view(-1, 1)
    count = s["row_start"][1:] - s["row_start"][:-1]
    s["lengths"] += count
    s["next_positions"] += count


def _plain_evict(s):
    c = s["c"]
    keep, page = c["keep"], c["page"]
    slots = s["scores"].shape[2]
    at = torch.arange(slots, device=DEV).view(1, 1, -1)
    length = s["lengths"].view(-1, 1, 1)
    held = (s["positions"] < c["sinks"]) | (s["positions"] >= (s["next_positions"] - c["recent"]).view(-1, 1, 1))
    key = torch.where(held, torch.full_like(s["scores"], math.inf), s["scores"])
    key = torch.where(at < length, key, torch.full_like(key, -1.0))
    best = torch.sort(key, dim=2, descending=True, stable=True).indices[:, :, :keep]
    kept = torch.zeros(key.shape, dtype=torch.bool, device=DEV).scatter_(2, best, True)
    full = length > keep
    hb, hh, dst = (full & ~kept & (at < keep)).nonzero(as_tuple=True)
    sb, sh, src = (full & kept & (at >= keep)).nonzero(as_tuple=True)
    to, frm = s["page_table"][hb, dst // page].long(), s["page_table"][sb, src // page].long()
    for pool in (s["k_pool"], s["v_pool"]):
        pool[to, hh, dst % page] = pool[frm, sh, src % page]
    s["scores"][hb, hh, dst] = s["scores"][sb, sh, src]
    s["positions"][hb, hh, dst] = s["positions"][sb, sh, src]
    if keep % page:                                           # the last kept page ends in zeros
        last = s["page_table"][full.view(-1), keep // page].long()
        s["k_pool"][last, :, keep % page:] = 0
        s["v_pool"][last, :, keep % page:] = 0
    s["lengths"].clamp_(max=keep)


# ---------------------------------------------------------------------------- one pass

def _handle(s):
    """What a program keeps beside its cache: the batch's description and a workspace."""
    if s["own"] is None:
        import transformer_kv_cache_b200 as kvc
        c = s["c"]
        batch = kvc.make_paged_batch(
            s["k_pool"], s["v_pool"], s["page_table"], s["lengths"], num_q_heads=c.get("hq", c["hkv"]),
            softmax_scale=s.get("scale", 1.0), prefix_pages=s["prefix_pages"] if c.get("prefix") else None,
            prefix_tokens=c.get("prefix", 0), next_positions=s.get("next_positions"), scores=s.get("scores"),
            positions=s.get("positions"))
        rows = s["q"].shape[0] if "q" in s else 0
        need = kvc.kvc_paged_workspace(batch, rows, c.get("keep", 0))
        s["own"] = kvc, batch, torch.empty(need, dtype=torch.uint8, device=DEV)
    return s["own"]


def run(s):
    c = s["c"]
    op = c["op"]
    if op == "attend":
        if not own:
            return _plain_attend(s)
        kvc, batch, work = _handle(s)
        kvc.kvc_paged_attend(batch, s["q"], s["o"], s["row_start"], work, lse=s["lse"], causal=c["causal"])
        return {"o": s["o"], "lse": s["lse"]}
    if op == "weights":
        if not own:
            return _plain_weights(s)
        kvc, batch, work = _handle(s)
        kvc.kvc_paged_weights(batch, s["q"], s["lse"], s["row_start"], work, causal=c["causal"])
        return {"scores": s["scores"]}
    if op == "append" or not c["n"]:
        # the drafts before these are taken back; or a new prompt's cache stands here
        s["lengths"].copy_(s["lengths0"])
        s["next_positions"].copy_(s["next0"])
        if op == "evict":
            s["scores"].copy_(s["scores0"])
            s["positions"].copy_(s["positions0"])
    if not own:
        if c["n"]:
            _plain_append(s)
        if op == "evict":
            _plain_evict(s)
    else:
        kvc, batch, work = _handle(s)
        if c["n"]:
            kvc.kvc_paged_append(batch, s["k"], s["v"], s["row_start"])
        if op == "evict":
            kvc.kvc_paged_evict(batch, c["keep"], c["sinks"], c["recent"], work)
    return {k: s[k] for k in ("k_pool", "v_pool", "lengths", "next_positions", "scores", "positions")}


def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    tokens, rows, row = sum(_lengths(c)), sum(_rows(c)), c["hkv"] * c["d"] * e
    if c["op"] in ("attend", "weights"):
        seen = 0
        for n, length in zip(sorted(_rows(c)), sorted(_lengths(c))):
            cut = n * (n - 1) // 2 if c["causal"] else 0
            seen += n * length - cut
        q = rows * c["hq"] * c["d"] * e
        if c["op"] == "attend":
            seen += rows * c["prefix"]
            return {"bytes": 2 * (tokens + c["prefix"]) * row + 2 * q + 4 * rows * c["hq"],
                    "flops": 4 * seen * c["hq"] * c["d"]}
        return {"bytes": tokens * row + q + 4 * rows * c["hq"] + 8 * tokens * c["hkv"],
                "flops": 2 * seen * c["hq"] * c["d"]}
    new = rows if c["n"] else 0
    entries = new * c["hkv"]
    total = 4 * new * row + 8 * entries if new else 0
    if c["op"] == "evict":
        before = tokens + new
        moved = 0
        for length in _lengths(c):
            length += c["n"]
            moved += c["n"] if c["n"] and c["n"] <= c["recent"] else c["keep"] * (length - c["keep"]) // length
        total += before * c["hkv"] * 8 + moved * (4 * row + 16 * c["hkv"])
    return {"bytes": total, "flops": 0}


# ---------------------------------------------------------------------------- in 64 bits

def _exact_state(case, seed):
    """Scores after an append and an eviction: one head at a time, from sorted tokens."""
    c = case
    s = prepare(c, seed)
    scores, positions = s["scores"].double().cpu().numpy(), s["positions"].cpu().numpy()
    starts, lengths, nexts = s["row_start"].tolist(), s["lengths"].tolist(), s["next_positions"].tolist()
    for b in range(c["b"]):
        new = starts[b + 1] - starts[b] if c["n"] else 0
        length, after = lengths[b] + new, nexts[b] + new
        scores[b, :, length - new:length] = 0.0
        positions[b, :, length - new:length] = np.arange(nexts[b], after)
        if c["op"] == "append" or length <= c["keep"]:
            continue
        for h in range(c["hkv"]):
            x, at = scores[b, h, :length], positions[b, h, :length]
            held = (at < c["sinks"]) | (at >= after - c["recent"])
            order = np.lexsort((np.arange(length), -x, ~held))[: c["keep"]]
            gone = np.setdiff1d(np.arange(c["keep"]), order)
            x[gone] = x[np.sort(order[order >= c["keep"]])]
    return {"k_pool": None, "v_pool": None, "lengths": None, "next_positions": None,
            "scores": torch.from_numpy(scores), "positions": None}


def exact(case, seed):
    if case["op"] in ("append", "evict"):
        return _exact_state(case, seed)
    c = case
    s = prepare(c, seed)
    g, page, scale = c["hq"] // c["hkv"], c["page"], 1.0 / math.sqrt(c["d"])
    starts, lengths = s["row_start"].tolist(), s["lengths"].tolist()
    attend = c["op"] == "attend"
    if attend:
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    else:
        scores = s["scores"].double()
    for b in range(c["b"]):
        r0, r1, length = starts[b], starts[b + 1], lengths[b]
        ids = [(int(p), page) for p in s["page_table"][b, : -(-length // page)]]
        before = c.get("prefix", 0)
        slots = torch.tensor([p for p, _ in ids], device=DEV, dtype=torch.long)
        for h in range(c["hkv"]):
            k = s["k_pool"][slots, h].reshape(-1, c["d"])[:length].double()
            if before:
                front = s["prefix_pages"].long()
                k = torch.cat([s["k_pool"][front, h].reshape(-1, c["d"])[:before].double(), k])
            q = s["q"][r0:r1, h * g:(h + 1) * g].double()                        # [n, g, d]
            x = torch.einsum("ngd,kd->ngk", q, k) * scale
            if c["causal"]:
                last = before + length - (r1 - r0) + torch.arange(r1 - r0, device=DEV)
                ahead = torch.arange(k.shape[0], device=DEV).view(1, 1, -1) > last.view(-1, 1, 1)
                x = torch.where(ahead, torch.full_like(x, -math.inf), x)
            if attend:
                v = s["v_pool"][slots, h].reshape(-1, c["d"])[:length].double()
                if before:
                    v = torch.cat([s["v_pool"][front, h].reshape(-1, c["d"])[:before].double(), v])
                lse[r0:r1, h * g:(h + 1) * g] = torch.logsumexp(x, -1)
                o[r0:r1, h * g:(h + 1) * g] = torch.einsum("ngk,kd->ngd", torch.softmax(x, -1), v)
            else:
                y = s["lse"][r0:r1, h * g:(h + 1) * g].double()
                scores[b, h, :length] += torch.exp(x - y.unsqueeze(-1)).sum((0, 1))
    return {"o": o, "lse": lse} if attend else {"scores": scores}
