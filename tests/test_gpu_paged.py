"""The paged-batch operators through the binding against fp64 (attention, weights) or
exactly (append, eviction): head layouts, types, page sizes, ragged rows, empty and
one-token sequences, masks that leave a row nothing, stale NaN in every unused slot."""
import copy
import math

import pytest
import torch

from paged_util import Batch, append_ref, attend64, evict_ref, weights64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import transformer_kv_cache_b200
    return transformer_kv_cache_b200


# rows, lengths, query heads, KV heads, head dim, page size, prefix, causal
SHAPES = {
    "one token": dict(rows=[1], lengths=[1], hq=1, hkv=1, d=64, causal=True),
    "one token behind a prefix of one": dict(rows=[1], lengths=[0], hq=2, hkv=2, d=64, prefix=1, causal=False),
    "decode, groups of 4": dict(rows=[1] * 5, lengths=[130, 1, 257, 64, 128], hq=8, hkv=2, d=128, prefix=300,
                                causal=True),
    "decode, groups of 7": dict(rows=[1, 1, 1], lengths=[700, 31, 5], hq=7, hkv=1, d=64, prefix=129, causal=True),
    "drafts, groups of 5": dict(rows=[3, 8, 1, 5], lengths=[40, 8, 300, 1000], hq=15, hkv=3, d=128, page=32, prefix=65,
                                causal=True),
    "empty sequences and rows": dict(rows=[2, 0, 3, 1, 0], lengths=[5, 17, 0, 0, 0], hq=4, hkv=4, d=64, causal=False),
    "rows that see nothing": dict(rows=[6, 4], lengths=[2, 0], hq=4, hkv=2, d=64, causal=True),
    "no own tokens": dict(rows=[4, 4], lengths=[0, 0], hq=4, hkv=2, d=128, prefix=47, causal=True),
    "frames, both ways": dict(rows=[150, 301], lengths=[333, 1290], hq=4, hkv=4, d=64, prefix=512, causal=False),
    "chunks, causal": dict(rows=[200, 77, 129], lengths=[200, 500, 130], hq=6, hkv=2, d=128, page=64, causal=True),
    "a long prompt, causal": dict(rows=[700], lengths=[1500], hq=2, hkv=1, d=64, page=128, prefix=40, causal=True),
    "pages of 256 that end inside": dict(rows=[1, 2, 9], lengths=[70, 200, 300], hq=8, hkv=4, d=64, page=256,
                                         prefix=333, causal=True),
    "groups of 64": dict(rows=[3, 1], lengths=[90, 400], hq=64, hkv=1, d=64, causal=True),
    "groups of 33": dict(rows=[7, 2], lengths=[90, 400], hq=66, hkv=2, d=128, prefix=20, causal=True),
    "many short sequences": dict(rows=[1 + i % 3 for i in range(400)], lengths=[3 + i % 41 for i in range(400)], hq=2,
                                 hkv=1, d=64, prefix=33, causal=True),
    "one long sequence": dict(rows=[1], lengths=[20011], hq=4, hkv=1, d=128, causal=True),
}
DTYPES = {"bf16": BF16, "f32": F32}
CASES = [(n, t) for n in SHAPES for t in DTYPES]
IDS = [f"{n}, {t}" for n, t in CASES]


def build(shape, dtype, **kw):
    s = dict(SHAPES[shape]) if isinstance(shape, str) else dict(shape)
    causal = s.pop("causal", True)
    return Batch(dtype=DTYPES[dtype], **{**s, **kw}), causal


def run_attend(kvc, t, causal, stream=None):
    c = copy.deepcopy(t).to(DEV)
    batch = c.handle(kvc)
    o = torch.full(c.q.shape, 7.0, dtype=c.dtype, device=DEV)
    lse = torch.full(c.q.shape[:2], 7.0, device=DEV)
    kvc.kvc_paged_attend(batch, c.q, o, c.row_start, c.workspace(kvc, batch), lse=lse, causal=causal, stream=stream)
    torch.cuda.synchronize()
    assert int(c.error) == 0
    return o.cpu(), lse.cpu()


def check_attend(t, causal, o, lse):
    ref, ref_lse, ob, lb = attend64(t, causal)
    total = int(t.row_start[-1])
    err = (o.double() - ref).abs()[:total]
    assert torch.isfinite(o.float()).all()
    assert (err <= ob[:total]).all(), (err / ob[:total]).max()
    none = torch.isinf(ref_lse[:total])
    assert torch.equal(torch.isinf(lse[:total]), none)
    err = (lse.double() - ref_lse)[:total].abs()
    assert (err[~none] <= lb[:total][~none]).all(), (err[~none] / lb[:total][~none]).max()
    # rows behind the last sequence are left as they were
    assert (o[total:].float() == 7).all() and (lse[total:] == 7).all()


@pytest.mark.parametrize("shape,dtype", CASES, ids=IDS)
def test_attend(kvc, shape, dtype):
    t, causal = build(shape, dtype, behind=3, seed=11)
    check_attend(t, causal, *run_attend(kvc, t, causal))


@pytest.mark.parametrize("shape,dtype", CASES, ids=IDS)
def test_weights(kvc, shape, dtype):
    t, causal = build(shape, dtype, behind=3, seed=12)
    _, lse, _, _ = attend64(t, causal)
    lse = lse.float()
    lse[-3:] = math.nan                                       # rows of nobody
    c = copy.deepcopy(t).to(DEV)
    batch = c.handle(kvc)
    work = c.workspace(kvc, batch)
    kvc.kvc_paged_weights(batch, c.q, lse.to(DEV), c.row_start, work, causal=causal)
    torch.cuda.synchronize()
    assert int(c.error) == 0
    ref, bound = weights64(t, lse, causal)
    got = c.scores.cpu().double()
    assert ((got - ref).abs() <= bound).all(), ((got - ref).abs() / bound.clamp_min(1e-300)).max()
    past = torch.arange(got.shape[2]).view(1, 1, -1) >= t.lengths.view(-1, 1, 1)
    past = past.expand_as(got)
    assert torch.equal(c.scores.cpu()[past], t.scores[past])  # slots past the length: untouched


# sequences around a warp's 32 and a block's 384 and 640 threads (who makes the schedule), every one of which
# ends inside a page of any size, with segments of one key tile and more, and rows that fill one tile or two
SCHEDULES = {
    "31 and a prefix": dict(rows=[1] * 31, lengths=[1 + 9 * i for i in range(31)], hq=8, hkv=2, d=128, page=256,
                            prefix=201),
    "32 and a prefix": dict(rows=[1 + i % 4 for i in range(32)], lengths=[5 + 11 * i for i in range(32)], hq=4, hkv=2,
                            d=64, page=128, prefix=77),
    "32": dict(rows=[2] * 32, lengths=[3 + 13 * i for i in range(32)], hq=6, hkv=2, d=128, page=64),
    "33": dict(rows=[1 + i % 3 for i in range(33)], lengths=[3 + 13 * i for i in range(33)], hq=6, hkv=2, d=64, page=32),
    "385": dict(rows=[1] * 385, lengths=[1 + (7 * i) % 150 for i in range(385)], hq=2, hkv=1, d=128, page=128, prefix=130),
    "650 of many rows": dict(rows=[1 + i % 2 for i in range(649)] + [90], lengths=[2 + i % 19 for i in range(649)] + [777],
                             hq=2, hkv=1, d=64, page=256, prefix=9),
    "17 to 32 rows of a head": dict(rows=[5, 6, 8, 7, 8], lengths=[300, 65, 8, 129, 1000], hq=12, hkv=3, d=128, page=32),
    "one row tile and two": dict(rows=[100, 130, 256, 257, 1], lengths=[500, 131, 256, 700, 90], hq=2, hkv=2, d=64,
                                 page=128, prefix=120),
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SCHEDULES)
def test_schedules(kvc, shape, dtype):
    """Attention and weights over batches whose schedules differ, both ways of masking."""
    for causal in (True, False):
        t, _ = build(SCHEDULES[shape], dtype, seed=31)
        o, lse = run_attend(kvc, t, causal)
        check_attend(t, causal, o, lse)
        c = copy.deepcopy(t).to(DEV)
        batch = c.handle(kvc)
        kvc.kvc_paged_weights(batch, c.q, lse.to(DEV), c.row_start, c.workspace(kvc, batch), causal=causal)
        torch.cuda.synchronize()
        assert int(c.error) == 0
        ref, bound = weights64(t, lse, causal)
        assert ((c.scores.cpu().double() - ref).abs() <= bound).all()


def test_weights_sum_to_the_rows(kvc):
    """Without a prefix every row's weights sum to 1: the scores gain rows x group in all."""
    t, causal = build("chunks, causal", "bf16", seed=3)
    t.scores.zero_()
    c = copy.deepcopy(t).to(DEV)
    batch = c.handle(kvc)
    work = c.workspace(kvc, batch)
    o, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device=DEV)
    kvc.kvc_paged_attend(batch, c.q, o, c.row_start, work, lse=lse, causal=causal)
    kvc.kvc_paged_weights(batch, c.q, lse, c.row_start, work, causal=causal)
    torch.cuda.synchronize()
    gain = c.scores.double().sum(2).cpu()
    want = torch.tensor(t.rows, dtype=torch.float64).view(-1, 1) * (t.hq // t.hkv)
    assert ((gain - want).abs() <= want * 2.0 ** -16).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_rows_of_a_fused_tensor(kvc, dtype):
    """Q, K and V as slices of one [rows, (hq + 2 hkv) d] tensor."""
    t, causal = build("drafts, groups of 5", dtype, seed=4, room=16)
    c = copy.deepcopy(t).to(DEV)
    g = torch.Generator().manual_seed(9)
    total = c.q.shape[0]
    fused = torch.randn(total, (t.hq + 2 * t.hkv) * t.d, generator=g).to(t.dtype).to(DEV)
    fused[:, : t.hq * t.d] = c.q.reshape(total, -1)
    q, k, v = fused.split([t.hq * t.d, t.hkv * t.d, t.hkv * t.d], 1)
    q, k, v = q.view(total, t.hq, t.d), k.view(total, t.hkv, t.d), v.view(total, t.hkv, t.d)
    assert not q.is_contiguous()
    batch = c.handle(kvc)
    kvc.kvc_paged_append(batch, k, v, c.row_start)
    o, lse = torch.empty(q.shape, dtype=t.dtype, device=DEV), torch.empty(q.shape[:2], device=DEV)
    kvc.kvc_paged_attend(batch, q, o, c.row_start, c.workspace(kvc, batch), lse=lse, causal=causal)
    torch.cuda.synchronize()
    append_ref(t, k.cpu(), v.cpu())
    check_attend(t, causal, o.cpu(), lse.cpu())


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_and_sharp_logits(kvc, dtype):
    """Logits of hundreds that grow along the keys, so the running maximum moves in every tile."""
    t, causal = build(dict(rows=[3, 1], lengths=[1000, 300], hq=4, hkv=2, d=64, prefix=400), dtype, seed=5)
    q = t.q.float()
    t.q = (q.abs() + 0.5).to(t.dtype)
    for b in range(t.b):
        n = int(t.lengths[b])
        at = torch.arange(n)
        ramp = (0.01 * at.float()).view(-1, 1, 1).expand(n, t.hkv, t.d).to(t.dtype)
        t.k_pool[t.page_table[b].long()[at // t.page], :, at % t.page] = ramp
    check_attend(t, causal, *run_attend(kvc, t, causal))


@pytest.mark.parametrize("dtype", DTYPES)
def test_hidden_infinities(kvc, dtype):
    """+-inf and the type's lowest value in slots past the length change nothing."""
    t, causal = build("pages of 256 that end inside", dtype, seed=6)
    want = run_attend(kvc, t, causal)
    for value in (math.inf, -math.inf, torch.finfo(t.dtype).min):
        u, _ = build("pages of 256 that end inside", dtype, seed=6, stale=value)
        got = run_attend(kvc, u, causal)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", DTYPES)
def test_page_outside_the_pool(kvc, dtype):
    """Such a page counts as zeros, an append skips it, and the error word tells."""
    t, causal = build(dict(rows=[2, 1], lengths=[100, 40], hq=4, hkv=2, d=64), dtype, seed=7)
    for bad in (-1, t.k_pool.shape[0], 2 ** 31 - 1, -2 ** 31):
        u = copy.deepcopy(t)
        page = int(u.page_table[0, 2])
        u.k_pool[page] = 0
        u.v_pool[page] = 0
        c = copy.deepcopy(t).to(DEV)
        c.page_table[0, 2] = bad
        batch = c.handle(kvc)
        work = c.workspace(kvc, batch, keep=20)
        o, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device=DEV)
        kvc.kvc_paged_attend(batch, c.q, o, c.row_start, work, lse=lse, causal=True)
        torch.cuda.synchronize()
        assert int(c.error) == 3
        check_attend(u, True, o.cpu(), lse.cpu())
        c.error.zero_()
        kvc.kvc_paged_weights(batch, c.q, lse, c.row_start, work)
        kvc.kvc_paged_evict(batch, 20, 0, 0, work)
        torch.cuda.synchronize()
        assert int(c.error) == 3 and c.lengths.tolist() == [20, 20]
        c.page_table[:] = bad
        before = c.k_pool.clone()
        c.error.zero_()
        kvc.kvc_paged_append(batch, c.q[:, :2], c.q[:, 2:], c.row_start)
        torch.cuda.synchronize()
        assert int(c.error) == 3
        assert torch.equal(before.view(torch.uint8), c.k_pool.view(torch.uint8))


def same_state(c, t, what):
    for name in ("k_pool", "v_pool"):
        a, b = getattr(c, name).cpu(), getattr(t, name)
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (what, name)
    for name in ("lengths", "next_positions", "positions"):
        assert torch.equal(getattr(c, name).cpu(), getattr(t, name)), (what, name)
    assert torch.equal(c.scores.cpu().view(torch.int32), t.scores.view(torch.int32)), (what, "scores")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,page,hkv", [(64, 16, 1), (128, 16, 8), (128, 64, 3), (64, 256, 2)])
def test_append(kvc, dtype, d, page, hkv):
    rows, lengths = [1, 0, 16, 5, 33, 2, 40], [0, 9, 16, 15, 1, 300, 290]
    t = Batch(rows=rows, lengths=lengths, hq=hkv, hkv=hkv, d=d, page=page, dtype=DTYPES[dtype], seed=1, room=20,
              behind=2)
    refused = [b for b in range(t.b) if rows[b] > t.max_pages * page - lengths[b]]
    assert refused == ([] if page == 256 else [6])            # the last does not fit
    c = copy.deepcopy(t).to(DEV)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(t.q.shape[0], hkv, d, generator=g).to(t.dtype) for _ in range(2))
    kvc.kvc_paged_append(c.handle(kvc), k.to(DEV), v.to(DEV), c.row_start)
    torch.cuda.synchronize()
    append_ref(t, k, v)
    same_state(c, t, "append")
    assert int(c.error) == (2 if refused else 0)


EVICTIONS = {
    "none over": dict(lengths=[10, 20], keep=20, sinks=1, recent=4),
    "one over": dict(lengths=[21, 20, 0], keep=20, sinks=1, recent=4),
    "to one": dict(lengths=[100, 1, 2], keep=1, sinks=0, recent=0),
    "all protected": dict(lengths=[100, 31, 33], keep=32, sinks=12, recent=20),
    "ragged": dict(lengths=[1000, 257, 511, 64, 2000], keep=200, sinks=4, recent=33),
    "half of a long one": dict(lengths=[9001], keep=4500, sinks=4, recent=100),
    "most of it": dict(lengths=[5000, 4097], keep=4096, sinks=0, recent=1),
    "eight and nine": dict(lengths=[108, 109, 101], keep=100, sinks=2, recent=10),
    "few of a long one": dict(lengths=[9003, 9000], keep=8999, sinks=2, recent=500),
    "few, and no slot to spare": dict(lengths=[24, 32], keep=24, sinks=24, recent=0),
}


@pytest.mark.parametrize("name", EVICTIONS)
@pytest.mark.parametrize("dtype,d,page,hkv", [("bf16", 64, 16, 4), ("bf16", 128, 32, 2), ("f32", 128, 64, 1)])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd values"])
def test_evict(kvc, name, dtype, d, page, hkv, kind):
    e = dict(EVICTIONS[name])
    lengths = e.pop("lengths")
    t = Batch(rows=[1] * len(lengths), lengths=lengths, hq=hkv, hkv=hkv, d=d, page=page, dtype=DTYPES[dtype], seed=3,
              stale=1.0)
    g = torch.Generator().manual_seed(4)
    t.scores = torch.exp(3 * torch.randn(t.scores.shape, generator=g))
    if kind == "ties":
        t.scores = torch.randint(0, 3, t.scores.shape, generator=g).float()
    elif kind == "odd values":
        odd = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-42, -1.0, 3e38])
        t.scores = odd[torch.randint(0, 8, t.scores.shape, generator=g)]
    # positions in no order, as earlier evictions leave them
    for b in range(t.b):
        for h in range(hkv):
            n = lengths[b]
            t.positions[b, h, :n] = torch.randperm(n + 7, generator=g)[:n].to(torch.int32)
    t.next_positions += 7
    c = copy.deepcopy(t).to(DEV)
    batch = c.handle(kvc)
    kvc.kvc_paged_evict(batch, e["keep"], e["sinks"], e["recent"], c.workspace(kvc, batch, e["keep"]))
    torch.cuda.synchronize()
    evict_ref(t, e["keep"], e["sinks"], e["recent"])
    same_state(c, t, name)
    assert int(c.error) == 0


def step_tensors(t, g, dev):
    total = sum(t.rows)
    return [torch.randn(total, h, t.d, generator=g).to(t.dtype).to(dev) for h in (t.hq, t.hkv, t.hkv)]


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_run_of_steps(kvc, dtype):
    """Append, attend, weigh, evict, step after step: attention and weights against fp64 on the
    cache as it stands, and the eviction exactly, from the scores that the library has."""
    rows, keep = [1, 3, 2], 96
    t = Batch(rows=rows, lengths=[90, 5, 96], hq=8, hkv=2, d=64, dtype=DTYPES[dtype], prefix=50, seed=8, room=8,
              stale=0.0)
    t.scores.zero_()
    c = copy.deepcopy(t).to(DEV)
    batch = c.handle(kvc)
    g = torch.Generator().manual_seed(10)
    for step in range(6):
        q, k, v = step_tensors(t, g, "cpu")
        t.q = q
        qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
        c.q = qd
        work = c.workspace(kvc, batch, keep)
        o, lse = torch.full(q.shape, 7.0, dtype=t.dtype, device=DEV), torch.full(q.shape[:2], 7.0, device=DEV)
        kvc.kvc_paged_append(batch, kd, vd, c.row_start)
        kvc.kvc_paged_attend(batch, qd, o, c.row_start, work, lse=lse)
        append_ref(t, k, v)
        check_attend(t, True, o.cpu(), lse.cpu())
        kvc.kvc_paged_weights(batch, qd, lse, c.row_start, work)
        ref, bound = weights64(t, lse.cpu(), True)
        assert ((c.scores.cpu().double() - ref).abs() <= bound).all()
        t.scores = c.scores.cpu()
        kvc.kvc_paged_evict(batch, keep, 4, 16, work)
        torch.cuda.synchronize()
        evict_ref(t, keep, 4, 16)
        same_state(c, t, step)
    assert int(c.error) == 0 and c.lengths.tolist() == [96, 23, 96]


def test_pages_serve_the_allocation_free_attention(kvc):
    """After an append and an eviction the pages hold zeros past the length, so
    kvc_attend_paged_noalloc reads them as they are."""
    t = Batch(rows=[20], lengths=[230], hq=4, hkv=4, d=64, seed=9, room=40, stale=0.0)
    c = copy.deepcopy(t).to(DEV)
    batch = c.handle(kvc)
    g = torch.Generator().manual_seed(10)
    q, k, v = step_tensors(t, g, DEV)
    work = c.workspace(kvc, batch, 203)
    kvc.kvc_paged_append(batch, k, v, c.row_start)
    kvc.kvc_paged_evict(batch, 203, 4, 30, work)
    kvc.kvc_paged_append(batch, k[:5].contiguous(), v[:5].contiguous(),
                         torch.tensor([0, 5], dtype=torch.int32, device=DEV))
    o1, o2 = torch.empty_like(q), torch.empty_like(q)
    kvc.kvc_paged_attend(batch, q, o1, c.row_start, work, causal=False)
    n = 208
    table = torch.zeros(-(-n // 16), 4, dtype=torch.int32)
    table[:, 0] = c.page_table[0, : table.shape[0]].cpu()
    table[:, 3] = 16
    kvc.kvc_attend_paged_noalloc(q, o2, c.k_pool, c.v_pool, c.k_pool.shape[0], table.to(DEV), table.shape[0], 20, 4, 64,
                                 16, t.scale)
    torch.cuda.synchronize()
    # both round their weights and their result to bf16 once
    bound = 4 * 2.0 ** -8 * c.v_pool.float().abs().max()
    assert (o1.float() - o2.float()).abs().max() <= bound


@pytest.mark.parametrize("dtype", DTYPES)
def test_graph_replays_follow_the_lengths(kvc, dtype):
    """One captured step, replayed: the same as the calls, whatever the lengths have become. Two
    graphs with a workspace each."""
    def fresh():
        t = Batch(rows=[1, 2], lengths=[120, 0], hq=4, hkv=2, d=64, dtype=DTYPES[dtype], prefix=40, seed=8, room=40,
                  stale=0.0)
        t.scores.zero_()
        return t.to(DEV)

    def step(c, batch, work, q, k, v, o, lse):
        kvc.kvc_paged_append(batch, k, v, c.row_start)
        kvc.kvc_paged_attend(batch, q, o, c.row_start, work, lse=lse)
        kvc.kvc_paged_weights(batch, q, lse, c.row_start, work)
        kvc.kvc_paged_evict(batch, 124, 2, 8, work)

    g = torch.Generator().manual_seed(3)
    base = fresh()
    ins = [step_tensors(base, g, DEV) for _ in range(8)]
    ref, got = fresh(), fresh()
    rb, gb = ref.handle(kvc), got.handle(kvc)
    rw, gw = ref.workspace(kvc, rb, 124), got.workspace(kvc, gb, 124)
    q, k, v = (x.clone() for x in ins[0])
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    o2, lse2 = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    warm = fresh()
    step(warm, warm.handle(kvc), warm.workspace(kvc, warm.handle(kvc), 124), q, k, v, o, lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(got, gb, gw, q, k, v, o, lse)
    for x in ins:
        for dst, src in zip((q, k, v), x):
            dst.copy_(src)
        graph.replay()
        step(ref, rb, rw, *x, o2, lse2)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert torch.equal(got.scores, ref.scores) and torch.equal(got.lengths, ref.lengths)
        assert torch.equal(got.positions, ref.positions)
        assert torch.equal(got.k_pool.view(torch.uint8), ref.k_pool.view(torch.uint8))


def test_two_streams_with_a_workspace_each(kvc):
    t, causal = build("decode, groups of 4", "bf16", seed=13)
    u, _ = build("frames, both ways", "bf16", seed=14)
    want = run_attend(kvc, t, causal), run_attend(kvc, u, False)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    cs, outs = [], []
    for x in (t, u):
        c = copy.deepcopy(x).to(DEV)
        b = c.handle(kvc)
        cs.append((c, b, c.workspace(kvc, b), torch.empty_like(c.q), torch.empty(c.q.shape[:2], device=DEV)))
    torch.cuda.synchronize()
    for _ in range(10):
        for (c, b, w, o, lse), s, cz in zip(cs, (s1, s2), (causal, False)):
            kvc.kvc_paged_attend(b, c.q, o, c.row_start, w, lse=lse, causal=cz, stream=s)
    torch.cuda.synchronize()
    for (c, b, w, o, lse), (wo, wl) in zip(cs, want):
        assert torch.equal(o.cpu(), wo) and torch.equal(lse.cpu(), wl)


def test_same_call_twice_gives_the_same_bits(kvc):
    for dtype in DTYPES:
        t, causal = build("drafts, groups of 5", dtype, seed=15)
        a, b = run_attend(kvc, t, causal), run_attend(kvc, t, causal)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_lengths_and_rows_out_of_range_are_reported(kvc):
    t, _ = build(dict(rows=[2, 1], lengths=[30, 16], hq=2, hkv=2, d=64), "bf16", seed=16)
    for change in ("long", "negative", "rows"):
        c = copy.deepcopy(t).to(DEV)
        if change == "long":
            c.lengths[0] = 10 ** 9
        elif change == "negative":
            c.lengths[1] = -5
        else:
            c.row_start[:] = torch.tensor([0, 2, 10 ** 6], dtype=torch.int32)
        batch = c.handle(kvc)
        work = c.workspace(kvc, batch, 8)
        o, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device=DEV)
        kvc.kvc_paged_attend(batch, c.q, o, c.row_start, work, lse=lse)
        torch.cuda.synchronize()
        assert int(c.error) == 3, change
        c.error.zero_()
        kvc.kvc_paged_weights(batch, c.q, torch.zeros_like(lse), c.row_start, work)
        torch.cuda.synchronize()
        assert int(c.error) == 3, change
        c.error.zero_()
        kvc.kvc_paged_append(batch, c.q, c.q, c.row_start)
        torch.cuda.synchronize()
        assert int(c.error) == 3, change


def test_log_sum_exp_that_is_no_number(kvc):
    """Rows with an LSE of +inf add exactly nothing; a NaN reaches the tokens that its row sees."""
    for dtype in DTYPES:
        t, _ = build(dict(rows=[64, 70], lengths=[200, 333], hq=4, hkv=2, d=64), dtype, seed=17)
        c = copy.deepcopy(t).to(DEV)
        batch = c.handle(kvc)
        work = c.workspace(kvc, batch)
        lse = torch.full(c.q.shape[:2], math.inf, device=DEV)
        kvc.kvc_paged_weights(batch, c.q, lse, c.row_start, work)
        torch.cuda.synchronize()
        assert torch.equal(c.scores.cpu(), t.scores)
        _, real, _, _ = attend64(t, True)
        lse = real.float().to(DEV)
        lse[64 + 5] = math.nan                                # row 5 of sequence 1
        kvc.kvc_paged_weights(batch, c.q, lse, c.row_start, work)
        torch.cuda.synchronize()
        bad = torch.isnan(c.scores.cpu())
        want = torch.zeros_like(bad)
        want[1, :, : 333 - 70 + 5 + 1] = True
        assert torch.equal(bad, want)


def test_not_a_number_stays_with_its_rows(kvc):
    """A NaN or infinite query makes its own output NaN and no other row's."""
    for dtype in DTYPES:
        t, causal = build("chunks, causal", dtype, seed=18)
        want = run_attend(kvc, t, causal)
        t.q[3, 1, 7] = math.nan
        t.q[250, 4, 0] = math.inf
        got = run_attend(kvc, t, causal)
        for x, y in zip(got, want):
            differ = torch.isnan(x)
            while differ.dim() > 2:
                differ = differ.any(-1)
            assert differ.nonzero().tolist() == [[3, 1], [250, 4]]
            keep = ~differ
            assert torch.equal(x[keep], y[keep])


def test_append_of_rows_far_behind(kvc):
    """A sequence whose rows stand behind 2^27 others in K and V (32 lanes a row: their number
    passes 32 bits). The rows before are nobody's, so that they are never touched."""
    skip, n = (1 << 27) + 5, 9
    if torch.cuda.mem_get_info()[0] < (skip + n) * 128 + (8 << 30):
        pytest.skip("needs 26 GB of device memory")
    t, _ = build(dict(rows=[n], lengths=[20], hq=1, hkv=1, d=64, room=n), "bf16", seed=21)
    c = copy.deepcopy(t).to(DEV)
    k = torch.empty(skip + n, 1, 64, dtype=BF16, device=DEV)
    k[skip:] = c.q
    kvc.kvc_paged_append(c.handle(kvc), k, k, c.row_start + skip)
    torch.cuda.synchronize()
    assert int(c.error) == 0 and c.lengths.tolist() == [20 + n]
    for slot in range(20, 20 + n):
        for pool in (c.k_pool, c.v_pool):
            assert torch.equal(pool[c.page_table[0, slot // 16], 0, slot % 16], c.q[slot - 20, 0])


def test_an_infinite_score_is_not_a_number(kvc):
    """One key with an infinite element: a row with a score of +inf (or 0 x inf) is NaN, as the
    softmax of the formula is; a row with -inf gives the key a weight of 0. The keys take the
    places of a tile in turn: exponentials of different places may be computed differently."""
    for dtype in DTYPES:
        for d in (64, 128):
            for key in (0, 13, 127, 128 + 46):
                t, _ = build(dict(rows=[200], lengths=[400], hq=2, hkv=1, d=d), dtype, seed=20)
                t.k_pool[t.page_table[0, key // 16], 0, key % 16, 0] = math.inf
                o, _ = run_attend(kvc, t, False)
                bad = torch.isnan(o)
                want = (t.q[:, :, :1] >= 0).expand_as(bad)
                assert torch.equal(bad, want), (dtype, d, key)


def test_no_rows_and_no_lse(kvc):
    t, causal = build("decode, groups of 4", "bf16", seed=19)
    want = run_attend(kvc, t, causal)
    c = copy.deepcopy(t).to(DEV)
    batch = c.handle(kvc)
    work = c.workspace(kvc, batch)
    o = torch.empty_like(c.q)
    kvc.kvc_paged_attend(batch, c.q, o, c.row_start, work, causal=causal)
    none = c.q[:0]
    zeros = torch.zeros_like(c.row_start)
    kvc.kvc_paged_attend(batch, none, none, zeros, work)
    kvc.kvc_paged_weights(batch, none, torch.empty(0, t.hq, device=DEV), zeros, work)
    kvc.kvc_paged_append(batch, none[:, : t.hkv].contiguous(), none[:, : t.hkv].contiguous(), zeros)
    torch.cuda.synchronize()
    assert torch.equal(o.cpu(), want[0])
    assert torch.equal(c.scores.cpu(), t.scores) and torch.equal(c.lengths.cpu(), t.lengths)


def test_pages_past_two_to_the_31_elements(kvc):
    """The last pages of a pool of 2.3 G elements give what the first ones of a small pool give."""
    t = Batch(rows=[2], lengths=[150], hq=16, hkv=8, d=128, seed=20, room=20, stale=0.0, prefix=30)
    small = copy.deepcopy(t).to(DEV)
    far = copy.deepcopy(t).to(DEV)
    pages, n = 140_000, t.k_pool.shape[0]
    for name in ("k_pool", "v_pool"):
        pool = torch.empty((pages,) + tuple(t.k_pool.shape[1:]), dtype=t.dtype, device=DEV)
        pool[-n:] = getattr(far, name)
        setattr(far, name, pool)
    far.page_table += pages - n
    far.prefix_pages += pages - n
    assert far.k_pool[:-n].numel() > 2 ** 31
    g = torch.Generator().manual_seed(2)
    q, k, v = step_tensors(t, g, DEV)
    results = []
    for c in (small, far):
        batch = c.handle(kvc)
        work = c.workspace(kvc, batch, 100)
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
        kvc.kvc_paged_append(batch, k, v, c.row_start)
        kvc.kvc_paged_attend(batch, q, o, c.row_start, work, lse=lse)
        kvc.kvc_paged_weights(batch, q, lse, c.row_start, work)
        kvc.kvc_paged_evict(batch, 100, 4, 16, work)
        torch.cuda.synchronize()
        assert int(c.error) == 0
        results.append((o, lse, c.scores, c.positions, c.k_pool[-n:].clone(), c.v_pool[-n:].clone()))
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seed", range(12))
def test_drawn_batches(kvc, dtype, seed):
    """Random layouts: attention, then its weights, against fp64."""
    g = torch.Generator().manual_seed(1000 + seed)
    pick = lambda *a: a[int(torch.randint(len(a), (1,), generator=g))]
    upto = lambda n: int(torch.randint(n + 1, (1,), generator=g))
    b, hkv, group = 1 + upto(8), pick(1, 2, 3, 4), pick(1, 2, 3, 5, 6, 8, 12, 17)
    most = pick(1, 7, 130, 400)
    lengths = [upto(pick(3, 60, 700, 2000)) for _ in range(b)]
    causal = bool(upto(1))
    t = Batch(rows=[upto(most) for _ in range(b - 1)] + [1 + upto(most)], lengths=lengths, hq=hkv * group, hkv=hkv,
              d=pick(64, 128), page=pick(16, 32, 64, 128, 256), prefix=pick(0, 0, 5, 128, 300, 1111),
              dtype=DTYPES[dtype], seed=seed, behind=upto(3))
    o, lse = run_attend(kvc, t, causal)
    check_attend(t, causal, o, lse)
    total = int(t.row_start[-1])
    lse[total:] = math.nan
    c = copy.deepcopy(t).to(DEV)
    batch = c.handle(kvc)
    kvc.kvc_paged_weights(batch, c.q, lse.to(DEV), c.row_start, c.workspace(kvc, batch), causal=causal)
    torch.cuda.synchronize()
    ref, bound = weights64(t, lse, causal)
    assert ((c.scores.cpu().double() - ref).abs() <= bound).all()
