"""Shared by the paged-batch tests: small random batches, their operators in fp64, and the
error bounds of the kernels' arithmetic."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24


def rounding(dtype) -> float:
    """The largest relative error of one rounding to the type: half a step."""
    return torch.finfo(dtype).eps / 2


class Batch:
    """A batch on the CPU (`dev` moves it): sequences with their own tokens in random pages, a
    shared prefix, ragged rows. Slots that hold no token are NaN in both pools: no result may
    depend on them."""

    def __init__(self, *, rows, lengths, hq, hkv, d, page=16, prefix=0, dtype=torch.bfloat16, seed=0, room=0,
                 behind=0, spread=2.0, stale=math.nan):
        g = torch.Generator().manual_seed(seed)
        self.hq, self.hkv, self.d, self.page, self.prefix, self.dtype = hq, hkv, d, page, prefix, dtype
        self.rows, self.b = list(rows), len(rows)
        self.max_pages = max(1, -(-(max(lengths) + room) // page))
        pp = -(-prefix // page)
        pages = self.b * self.max_pages + pp + 2
        order = torch.randperm(pages, generator=g).to(torch.int32)
        self.prefix_pages = order[:pp].contiguous()
        self.page_table = order[pp:pp + self.b * self.max_pages].view(self.b, -1).contiguous()
        self.lengths = torch.tensor(lengths, dtype=torch.int32)
        self.row_start = torch.tensor([0] + torch.tensor(self.rows).cumsum(0).tolist(), dtype=torch.int32)
        total = sum(self.rows)
        self.q = (spread * torch.randn(total + behind, hq, d, generator=g)).to(dtype)
        self.k_pool = torch.full((pages, hkv, page, d), stale, dtype=dtype)
        self.v_pool = self.k_pool.clone()
        for ids, n in [(self.prefix_pages, prefix)] + [(self.page_table[b], lengths[b]) for b in range(self.b)]:
            for pool in (self.k_pool, self.v_pool):
                at = torch.arange(n)
                pool[ids[at // page].long(), :, at % page] = torch.randn(n, hkv, d, generator=g).to(dtype)
        slots = self.max_pages * page
        self.scores = torch.rand(self.b, hkv, slots, generator=g)
        self.positions = torch.arange(slots, dtype=torch.int32).expand(self.b, hkv, -1).contiguous()
        self.next_positions = self.lengths.clone()
        self.error = torch.zeros(1, dtype=torch.int32)
        self.scale = d ** -0.5

    ARRAYS = ("prefix_pages", "page_table", "lengths", "row_start", "q", "k_pool", "v_pool", "scores", "positions",
              "next_positions", "error")

    def to(self, dev):
        for n in self.ARRAYS:
            setattr(self, n, getattr(self, n).to(dev))
        return self

    def handle(self, kvc):
        return kvc.make_paged_batch(
            self.k_pool, self.v_pool, self.page_table, self.lengths, self.hq, self.scale,
            prefix_pages=self.prefix_pages if self.prefix else None, prefix_tokens=self.prefix,
            next_positions=self.next_positions, scores=self.scores, positions=self.positions, error=self.error)

    def workspace(self, kvc, batch, keep=0):
        # ff bytes: NaN as fp32 and negative as integers, so nothing may rely on zeros
        n = kvc.kvc_paged_workspace(batch, self.q.shape[0], keep)
        return torch.full((n,), 255, dtype=torch.uint8, device=self.q.device)

    def own(self, pool, b, h):
        n = int(self.lengths[b])
        ids = self.page_table[b].long()[: -(-n // self.page)]
        return pool[ids, h].reshape(-1, self.d)[:n].double()

    def front(self, pool, h):
        return pool[self.prefix_pages.long(), h].reshape(-1, self.d)[: self.prefix].double()


def heads_of(t, b, h):
    """Rows and query heads of sequence b's KV head h."""
    g = t.hq // t.hkv
    return slice(int(t.row_start[b]), int(t.row_start[b + 1])), slice(h * g, (h + 1) * g)


def seen(t, b, causal, before, n_keys):
    """[n, keys] which keys (prefix first) each row of sequence b sees."""
    n = t.rows[b]
    own = torch.arange(n_keys - before).view(1, -1)
    last = int(t.lengths[b]) - (n - 1 - torch.arange(n)).view(-1, 1) if causal else torch.full((n, 1), 1 << 30)
    ok = own < last if causal else own >= 0
    return torch.cat([torch.ones(n, before, dtype=torch.bool), ok.expand(n, -1)], 1)


def attend64(t, causal):
    """(O, LSE, bound of O's error, bound of the LSE's) in fp64. The bounds: a logit is a sum of
    D products in fp32 (or in a tensor core's fp32 accumulator, which may truncate: twice a
    rounding each) scaled once, so it is within d = 4 (D + 2) u A of the exact one, A the sum of
    the products' magnitudes; a weight is within e^(2 d) - 1 plus 2^-21 of the exponential's
    approximation, relatively, and for bf16 half a bf16 step on its way into the second
    product; sums of n terms add 2 n u; the result is rounded once to the output type."""
    o = torch.zeros(t.q.shape, dtype=torch.float64)
    lse = torch.zeros(t.q.shape[:2], dtype=torch.float64)
    ob, lb = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(t.b):
        for h in range(t.hkv):
            rs, hs = heads_of(t, b, h)
            k = torch.cat([t.front(t.k_pool, h), t.own(t.k_pool, b, h)])
            v = torch.cat([t.front(t.v_pool, h), t.own(t.v_pool, b, h)])
            q = t.q[rs, hs].double()
            if q.shape[0] == 0:
                continue
            x = torch.einsum("ngd,kd->ngk", q, k) * t.scale
            a = torch.einsum("ngd,kd->ngk", q.abs(), k.abs()) * t.scale
            ok = seen(t, b, causal, t.prefix, k.shape[0]).unsqueeze(1)
            x = torch.where(ok, x, torch.full_like(x, -math.inf))
            a = torch.where(ok, a, torch.zeros_like(a))
            none = ~ok.any(-1).expand(x.shape[:2])
            p = torch.exp(x - x.amax(-1, keepdim=True).clamp_min(-1e300)) if k.shape[0] else x
            s = p.sum(-1)
            p = torch.where(s.unsqueeze(-1) > 0, p / s.unsqueeze(-1).clamp_min(1e-300), torch.zeros_like(p))
            oo = torch.einsum("ngk,kd->ngd", p, v)
            ll = torch.where(none, torch.full_like(s, -math.inf),
                             torch.logsumexp(x, -1) if k.shape[0] else torch.full_like(s, -math.inf))
            o[rs, hs], lse[rs, hs] = oo, ll
            n = k.shape[0]
            amax = a.amax(-1) if n else torch.zeros(x.shape[:2], dtype=torch.float64)
            d = 4 * (t.d + 2) * U32 * amax
            e = torch.expm1(2 * d) + 2.0 ** -21 + 2 * n * U32
            w = e * 2 + (rounding(t.dtype) if t.dtype != torch.float32 else 0.0)
            # |sum p v| weights each value's magnitude by its own weight
            mass = torch.einsum("ngk,kd->ngd", p, v.abs())
            ob[rs, hs] = w.unsqueeze(-1) * mass * 1.01 + rounding(t.dtype) * oo.abs() * 1.01 + 1e-30
            lb[rs, hs] = 2 * d + e + 4 * U32 * torch.where(none, torch.zeros_like(ll), ll.abs()) + 2.0 ** -21
    return o, lse, ob, lb


def weights64(t, lse, causal):
    """(scores after the call, bound of their error) in fp64, given the LSE the call gets."""
    out, bound = t.scores.double().clone(), torch.zeros(t.scores.shape, dtype=torch.float64)
    for b in range(t.b):
        n = int(t.lengths[b])
        for h in range(t.hkv):
            rs, hs = heads_of(t, b, h)
            k, q = t.own(t.k_pool, b, h), t.q[rs, hs].double()
            if q.shape[0] == 0 or n == 0:
                continue
            y = lse[rs, hs].double()
            x = torch.einsum("ngd,kd->ngk", q, k) * t.scale
            a = torch.einsum("ngd,kd->ngk", q.abs(), k.abs()) * t.scale
            ok = seen(t, b, causal, 0, n).unsqueeze(1).expand_as(x)
            w = torch.where(ok, torch.exp(x - y.unsqueeze(-1)), torch.zeros_like(x))
            fin = torch.where(torch.isfinite(y), y.abs(), torch.zeros_like(y)).unsqueeze(-1)
            d = 4 * (t.d + 2) * U32 * a + 4 * U32 * (fin + a)
            terms = q.shape[0] * q.shape[1] + 2
            out[b, h, :n] += w.sum((0, 1))
            bound[b, h, :n] = (w * (torch.expm1(2 * d) + 2.0 ** -21 + 2 * terms * U32)).sum((0, 1))
    return out, bound + 4 * U32 * out.abs()


def append_ref(t, k, v):
    """The append, token by token, in place."""
    cap = t.max_pages * t.page
    for b in range(t.b):
        n, r0 = t.rows[b], int(t.row_start[b])
        if n > cap - int(t.lengths[b]):
            continue
        for i in range(n):
            slot = int(t.lengths[b])
            page = int(t.page_table[b, slot // t.page])
            if slot % t.page == 0:
                t.k_pool[page] = 0
                t.v_pool[page] = 0
            t.k_pool[page, :, slot % t.page] = k[r0 + i]
            t.v_pool[page, :, slot % t.page] = v[r0 + i]
            t.scores[b, :, slot] = 0
            t.positions[b, :, slot] = t.next_positions[b]
            t.lengths[b] += 1
            t.next_positions[b] += 1


def evict_ref(t, keep, sinks, recent):
    """The eviction, one head at a time, in place."""
    for b in range(t.b):
        n = int(t.lengths[b])
        if n <= keep:
            continue
        start = int(t.next_positions[b]) - recent
        for h in range(t.hkv):
            s, pos = t.scores[b, h], t.positions[b, h]

            def rank(j):
                held = int(pos[j]) < sinks or int(pos[j]) >= start
                x = float(s[j])
                return (not held, math.isnan(x), 0.0 if math.isnan(x) or held else -x, j)
            kept = set(sorted(range(n), key=rank)[:keep])
            to = [j for j in range(keep) if j not in kept]
            frm = [j for j in range(keep, n) if j in kept]
            for a, c in zip(frm, to):
                pa, pc = int(t.page_table[b, a // t.page]), int(t.page_table[b, c // t.page])
                for pool in (t.k_pool, t.v_pool):
                    pool[pc, h, c % t.page] = pool[pa, h, a % t.page]
                s[c], pos[c] = s[a].clone(), pos[a].clone()
        if keep % t.page:
            last = int(t.page_table[b, keep // t.page])
            t.k_pool[last, :, keep % t.page:] = 0
            t.v_pool[last, :, keep % t.page:] = 0
        t.lengths[b] = keep
