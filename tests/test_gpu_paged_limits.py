"""The paged-batch operators at the ends of their ranges: terms and scores that overflow, batches whose
rows are dealt out unevenly, and the forms that only large or full sequences take."""
import copy
import math

import pytest
import torch

from paged_util import Batch, append_ref, attend64, evict_ref, weights64
from test_gpu_paged import DEV, DTYPES, check_attend, run_attend, same_state, step_tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import transformer_kv_cache_b200
    return transformer_kv_cache_b200


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [64, 160])
def test_terms_around_the_largest_number(kvc, dtype, rows):
    """Weights with an LSE of the caller's: one row of each sequence, at a place of its own, has terms of
    2^127.5 (finite), of 2^130 (infinite) or of a product that is no number (no finite score), the
    others add nothing. 64 rows a sequence fit one tile, 160 do not: two forms of the bf16 kernel."""
    b, n = 32, 300
    for kind in ("finite", "infinite", "nan"):
        t = Batch(rows=[rows] * b, lengths=[n] * b, hq=1, hkv=1, d=64, dtype=DTYPES[dtype], seed=2)
        t.q.zero_()
        t.scores.zero_()
        lse = torch.full(t.q.shape[:2], 1000.0)
        hot = torch.tensor([rows * i + (rows - 32) * (i % 2) + i for i in range(b)])
        lse[hot] = {"finite": -127.5, "infinite": -130.0, "nan": 0.0}[kind] * math.log(2)
        if kind == "nan":
            t.q[hot, :, 5] = math.nan
        c = copy.deepcopy(t).to(DEV)
        batch = c.handle(kvc)
        kvc.kvc_paged_weights(batch, c.q, lse.to(DEV), c.row_start, c.workspace(kvc, batch), causal=False)
        torch.cuda.synchronize()
        got = c.scores.cpu()[:, :, :n].double()
        if kind == "finite":
            ref, bound = weights64(t, lse, False)
            assert ((got - ref[:, :, :n]).abs() <= bound[:, :, :n]).all(), got[:, 0, 0]
        elif kind == "infinite":
            assert (got == math.inf).all(), got[:, 0, 0]
        else:
            assert not torch.isfinite(got).any(), got[:, 0, 0]


def append_inputs(t):
    g = torch.Generator().manual_seed(2)
    return [torch.randn(t.q.shape[0], t.hkv, t.d, generator=g).to(t.dtype) for _ in range(2)]


def check_append(kvc, t, error, change=None):
    """The whole state after an append, against the append token by token; `change` is applied to the
    device's copy alone."""
    c = copy.deepcopy(t).to(DEV)
    if change:
        change(c)
    k, v = append_inputs(t)
    kvc.kvc_paged_append(c.handle(kvc), k.to(DEV), v.to(DEV), c.row_start)
    torch.cuda.synchronize()
    append_ref(t, k, v)
    assert int(c.error) == error
    return c


# a few rows a sequence and many, and a batch of one chunk among single rows
APPENDS = {
    "a few rows": dict(rows=[1, 0, 8, 5, 3, 7, 2, 16], lengths=[0, 9, 16, 15, 1, 300, 250, 31]),
    "single rows": dict(rows=[1] * 9, lengths=[0, 1, 15, 16, 17, 63, 64, 255, 256]),
    "a chunk among single rows": dict(rows=[1] * 30 + [200], lengths=[7 * i for i in range(31)]),
    "many rows": dict(rows=[40, 0, 17, 90], lengths=[0, 5, 47, 200]),
    "a row of a frame each": dict(rows=[1] * 700, lengths=[i % 50 for i in range(700)]),
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,page,hkv", [(64, 16, 1), (128, 64, 3), (64, 128, 8), (128, 256, 2)])
@pytest.mark.parametrize("name", APPENDS)
def test_append_forms(kvc, name, dtype, d, page, hkv):
    t = Batch(**APPENDS[name], hq=hkv, hkv=hkv, d=d, page=page, dtype=DTYPES[dtype], seed=1, room=200, behind=2)
    c = check_append(kvc, t, 0)
    same_state(c, t, name)


@pytest.mark.parametrize("rows", [[3, 1, 6, 2], [30, 1, 40, 2]], ids=["a few rows", "many rows"])
@pytest.mark.parametrize("page", [16, 256])
def test_append_takes_a_sequence_whole_or_not_at_all(kvc, rows, page):
    """No room, a length out of range, a next position out of range: that sequence takes nothing, the
    others all of theirs."""
    def fresh(room):
        return Batch(rows=rows, lengths=[250, 3, 256 - rows[2], 9], hq=2, hkv=2, d=64, page=page, seed=1, room=room)

    t = fresh(0)                                              # 256 slots: the first has no room, the third just enough
    t.lengths[0] = 256 - rows[0] + 1
    c = check_append(kvc, t, 2)
    same_state(c, t, "room")
    assert c.lengths.tolist()[0] == 256 - rows[0] + 1 and c.lengths.tolist()[2] == 256
    for length in (-1, -2 ** 31, 2 ** 31 - 1, 10 ** 9):
        t = fresh(64)
        keep = int(t.lengths[1])
        t.lengths[1] = 1 << 30                                # the reference takes nothing here either

        def change(c):
            c.lengths[1] = length
        c = check_append(kvc, t, 3, change)
        assert int(c.lengths[1]) == length
        c.lengths[1] = t.lengths[1] = keep
        same_state(c, t, length)
    for start in (2 ** 31 - rows[0], 2 ** 31 - 1):            # the first position past 32 bits, and all of them
        t = fresh(64)
        t.next_positions[0] = start
        n = t.rows[0]
        t.rows[0] = 0                                         # for the reference
        c = check_append(kvc, t, 3)
        t.rows[0] = n
        same_state(c, t, start)
    t = fresh(64)
    t.next_positions[0] = 2 ** 31 - 1 - rows[0]               # the last that fits
    c = check_append(kvc, t, 0)
    same_state(c, t, "last positions")


def evict_sorted(t, keep, sinks, recent):
    """evict_ref for long sequences and scores that are numbers: one sort a head."""
    slots = torch.arange(t.scores.shape[2])
    for b in range(t.b):
        n = int(t.lengths[b])
        if n <= keep:
            continue
        table = t.page_table[b].long()
        start = int(t.next_positions[b]) - recent
        for h in range(t.hkv):
            s, pos = t.scores[b, h, :n], t.positions[b, h, :n]
            held = (pos < sinks) | (pos >= start)
            key = torch.where(held, torch.full_like(s, math.inf), s)
            kept = torch.zeros(n, dtype=torch.bool)
            kept[torch.sort(key, descending=True, stable=True).indices[:keep]] = True
            to, frm = slots[:keep][~kept[:keep]], slots[keep:n][kept[keep:]]
            for pool in (t.k_pool, t.v_pool):
                pool[table[to // t.page], h, to % t.page] = pool[table[frm // t.page], h, frm % t.page]
            s[to], pos[to] = s[frm], pos[frm]
        if keep % t.page:
            for pool in (t.k_pool, t.v_pool):
                pool[table[keep // t.page], :, keep % t.page:] = 0
        t.lengths[b] = keep


# one head's slots in a cluster of 1, 2, 4 and 8 CTAs, and all that a cluster of 8 holds
CLUSTERS = {"1": 8192, "2": 8208, "4": 16400, "8": 32784, "8, full": 393216}


@pytest.mark.parametrize("cap", CLUSTERS.values(), ids=CLUSTERS)
@pytest.mark.parametrize("gone", [1, 8, 9, "half"])
@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_evict_in_clusters(kvc, cap, gone, kind):
    n = cap - 3
    keep = n // 2 if gone == "half" else n - gone
    t = Batch(rows=[1], lengths=[n], hq=1, hkv=1, d=64, seed=3, room=3, stale=1.0)
    assert t.max_pages * t.page == cap
    g = torch.Generator().manual_seed(4)
    # ties: few scores, so that runs of equal ones lie in every CTA of the cluster
    t.scores = torch.exp(3 * torch.randn(t.scores.shape, generator=g)) if kind == "spread" else \
        torch.randint(0, 3, t.scores.shape, generator=g).float()
    t.positions[0, 0, :n] = torch.randperm(n + 7, generator=g)[:n].to(torch.int32)
    t.next_positions += 7
    u = copy.deepcopy(t)
    c = copy.deepcopy(t).to(DEV)
    batch = c.handle(kvc)
    kvc.kvc_paged_evict(batch, keep, 4, 100, c.workspace(kvc, batch, keep))
    torch.cuda.synchronize()
    evict_sorted(t, keep, 4, 100)
    same_state(c, t, cap)
    assert int(c.error) == 0
    if cap == 8192 and gone != "half":                        # the sort against the plain reference
        evict_ref(u, keep, 4, 100)
        same_state(u, t, "references")


def test_pages_cut_inside_serve_the_allocation_free_attention(kvc):
    """A sequence that an eviction cut and an append continued ends inside a page whose other slots
    are zeros, in a pool that holds NaN wherever nothing was written: kvc_attend_paged_noalloc, which
    reads whole pages, gives the same attention."""
    rows, keep, n = 20, 203, 205
    t = Batch(rows=[rows], lengths=[230], hq=4, hkv=4, d=64, seed=9, room=40)
    c = copy.deepcopy(t).to(DEV)
    batch = c.handle(kvc)
    g = torch.Generator().manual_seed(10)
    q, k, v = step_tensors(t, g, "cpu")
    t.q = q
    start, two = c.row_start.clone(), torch.tensor([0, 2], dtype=torch.int32)
    work = c.workspace(kvc, batch, keep)
    kvc.kvc_paged_append(batch, k.to(DEV), v.to(DEV), c.row_start)
    kvc.kvc_paged_evict(batch, keep, 4, 30, work)
    kvc.kvc_paged_append(batch, k[:2].to(DEV), v[:2].to(DEV), two.to(DEV))
    append_ref(t, k, v)
    evict_ref(t, keep, 4, 30)
    t.rows, t.row_start = [2], two
    append_ref(t, k[:2], v[:2])
    t.rows, t.row_start = [rows], start.cpu()
    qd = q.to(DEV)
    o1, lse, o2 = torch.empty_like(qd), torch.empty(q.shape[:2], device=DEV), torch.empty_like(qd)
    kvc.kvc_paged_attend(batch, qd, o1, start, work, lse=lse, causal=False)
    table = torch.zeros(-(-n // 16), 4, dtype=torch.int32)
    table[:, 0] = t.page_table[0, : table.shape[0]]
    table[:, 3] = 16
    table[-1, 3] = n % 16
    kvc.kvc_attend_paged_noalloc(qd, o2, c.k_pool, c.v_pool, c.k_pool.shape[0], table.to(DEV), table.shape[0], rows, 4,
                                 64, 16, t.scale)
    torch.cuda.synchronize()
    same_state(c, t, "state")
    check_attend(t, False, o1.cpu(), lse.cpu())
    ref, _, bound, _ = attend64(t, False)
    # the library's frame attention adds up the weights that it has rounded to bf16, half a step (2^-8)
    # of each, and its exponential is a cubic of 1.02e-4, in the weights and in their sum: 2^-8 + 2.04e-4 <
    # 1.06 x 2^-8 of the values' mean magnitude more than `bound`, which holds 2^-8 of it already
    assert ((o2.cpu().double() - ref).abs() <= 2.06 * bound).all()


# one chunk among single rows, in numbers for which the average picks the form that suits neither
UNEVEN = {
    "the prefix read by every item": dict(rows=[1] * 15 + [1100], lengths=[40 + 9 * i for i in range(15)] + [1101], hq=8,
                                          hkv=2, d=64, prefix=333),
    "the prefix read by every item, 128 dims": dict(rows=[1] * 7 + [530], lengths=[3 + 31 * i for i in range(7)] + [700],
                                                    hq=4, hkv=1, d=128, page=32, prefix=130),
    "a chunk in tiles of few rows": dict(rows=[1] * 30 + [180], lengths=[10 * i for i in range(1, 31)] + [500], hq=2,
                                         hkv=2, d=64, page=64, prefix=77),
    "a chunk of several tiles": dict(rows=[1] * 10 + [700] + [1] * 10, lengths=[10 * i + 1 for i in range(10)] + [900] +
                                     [300] * 10, hq=2, hkv=1, d=128, prefix=0),
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", UNEVEN)
def test_a_chunk_among_single_rows(kvc, name, dtype):
    t = Batch(**UNEVEN[name], dtype=DTYPES[dtype], seed=5, behind=3)
    for causal in (True, False):
        o, lse = run_attend(kvc, t, causal)
        check_attend(t, causal, o, lse)
        c = copy.deepcopy(t).to(DEV)
        batch = c.handle(kvc)
        kvc.kvc_paged_weights(batch, c.q, lse.to(DEV), c.row_start, c.workspace(kvc, batch), causal=causal)
        torch.cuda.synchronize()
        assert int(c.error) == 0
        ref, bound = weights64(t, lse, causal)
        assert ((c.scores.cpu().double() - ref).abs() <= bound).all()


def in_guarded_memory(t):
    """The batch on the device with its pools, scores and positions as parts of one buffer, between bytes
    of 0x5a; and what gives the bytes that no array has."""
    names = ("k_pool", "v_pool", "scores", "positions")
    c = copy.deepcopy(t)
    at, gap = {}, 1 << 16
    end = gap
    for name in names:
        x = getattr(c, name)
        at[name] = end
        end += (x.numel() * x.element_size() + 255) // 256 * 256 + gap
    buf = torch.full((end,), 0x5a, dtype=torch.uint8, device=DEV)
    free = torch.ones(end, dtype=torch.bool, device=DEV)
    views = {}
    for name in names:
        x = getattr(c, name)
        n = x.numel() * x.element_size()
        views[name] = buf[at[name]:at[name] + n].view(x.dtype).view(x.shape)
        views[name].copy_(x)
        free[at[name]:at[name] + n] = False
        setattr(c, name, torch.empty(0))
    c.to(DEV)
    for name in names:
        setattr(c, name, views[name])
    return c, lambda: buf[free]


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_workspace_shared_by_mistake_stays_a_mistake_of_numbers(kvc, dtype):
    """Two batches of different sizes whose calls run at the same time with one workspace, which the
    header forbids: their numbers may be wrong, but nothing outside of their arrays is touched."""
    small = Batch(rows=[3, 1, 200], lengths=[700, 900, 1000], hq=4, hkv=2, d=64, prefix=100, dtype=DTYPES[dtype], seed=1,
                  stale=0.0)
    large = Batch(rows=[1, 2] * 20 + [300], lengths=[400 + 50 * i for i in range(40)] + [3000], hq=8, hkv=8, d=64, page=32,
                  dtype=DTYPES[dtype], seed=2, stale=0.0)
    keep = 150
    calls, works = [], []
    for t in (small, large):
        c, outside = in_guarded_memory(t)
        b = c.handle(kvc)
        works.append(c.workspace(kvc, b, keep))
        calls.append((c, b, outside, c.lengths.clone(), c.scores.clone(), torch.empty_like(c.q),
                      torch.empty(c.q.shape[:2], device=DEV), torch.cuda.Stream()))
    work = max(works, key=lambda w: w.numel())
    torch.cuda.synchronize()
    for i in range(60):
        for c, b, _, lengths, scores, o, lse, s in calls if i % 2 else calls[::-1]:
            with torch.cuda.stream(s):
                c.lengths.copy_(lengths)
                c.scores.copy_(scores)
                kvc.kvc_paged_attend(b, c.q, o, c.row_start, work, lse=lse)
                kvc.kvc_paged_weights(b, c.q, lse, c.row_start, work)
                kvc.kvc_paged_evict(b, keep, 4, 16, work)
    torch.cuda.synchronize()
    for c, _, outside, *_ in calls:
        assert (outside() == 0x5a).all()
        assert c.lengths.tolist() == [keep] * c.b
    # and with a workspace each the same arrays still give what they should
    for (c, b, _, lengths, scores, o, lse, _), w, t in zip(calls, works, (small, large)):
        c.lengths.copy_(lengths)
        for name in ("k_pool", "v_pool"):
            getattr(c, name).copy_(getattr(t, name))
        kvc.kvc_paged_attend(b, c.q, o, c.row_start, w, lse=lse, causal=True)
        torch.cuda.synchronize()
        check_attend(t, True, o.cpu(), lse.cpu())


def test_workspace_serves_fewer_rows(kvc):
    """The workspace for some rows is enough for every smaller number, and one that is too small is
    refused."""
    for dtype in DTYPES:
        for b, hq, hkv, d, prefix in ((1, 1, 1, 64, 0), (7, 8, 2, 64, 100), (64, 32, 8, 128, 5), (3, 64, 1, 128, 1000)):
            t = Batch(rows=[1] * b, lengths=[20] * b, hq=hq, hkv=hkv, d=d, prefix=prefix, dtype=DTYPES[dtype], seed=1).to(DEV)
            batch = t.handle(kvc)
            sizes = [kvc.kvc_paged_workspace(batch, n) for n in list(range(1200)) + [4096, 8191, 8192]]
            assert sizes == sorted(sizes)
        o, lse = torch.empty_like(t.q), torch.empty(t.q.shape[:2], device=DEV)
        small = torch.empty(256, dtype=torch.uint8, device=DEV)
        for call in (lambda: kvc.kvc_paged_attend(batch, t.q, o, t.row_start, small, lse=lse),
                     lambda: kvc.kvc_paged_weights(batch, t.q, lse, t.row_start, small),
                     lambda: kvc.kvc_paged_evict(batch, 8, 0, 0, small)):
            with pytest.raises(kvc.KVCError):
                call()
        torch.cuda.synchronize()
        assert int(t.error) == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_graph_replays_follow_rows_and_tables(kvc, dtype):
    """A captured attention and its weights, replayed for other row starts (none at all among them), other
    lengths and other pages."""
    t = Batch(rows=[100, 20, 24], lengths=[300, 90, 700], hq=4, hkv=2, d=64, prefix=70, dtype=DTYPES[dtype], seed=3)
    c = copy.deepcopy(t).to(DEV)
    batch = c.handle(kvc)
    work = c.workspace(kvc, batch)
    o, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device=DEV)

    def step():
        kvc.kvc_paged_attend(batch, c.q, o, c.row_start, work, lse=lse)
        kvc.kvc_paged_weights(batch, c.q, lse, c.row_start, work)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rows, lengths, swap in (([100, 20, 24], [300, 90, 700], False), ([1, 1, 1], [300, 90, 700], True),
                                ([0, 0, 0], [300, 90, 700], False), ([0, 144, 0], [300, 50, 0], False),
                                ([140, 0, 3], [1, 0, 700], True)):
        u = copy.deepcopy(t)
        u.rows, u.lengths = rows, torch.tensor(lengths, dtype=torch.int32)
        u.row_start = torch.tensor([0] + torch.tensor(rows).cumsum(0).tolist(), dtype=torch.int32)
        if swap:                                              # the first sequence's tokens in other pages
            n = -(-300 // 16)
            new = t.page_table[2, torch.arange(n) + 44 - n].flip(0).clone()      # of the third's last ones
            u.k_pool[new.long()], u.v_pool[new.long()] = (p[t.page_table[0, :n].long()] for p in (t.k_pool, t.v_pool))
            u.page_table[0, :n] = new
            u.lengths[2] = min(int(u.lengths[2]), (44 - n) * 16)
        for name in ("lengths", "row_start", "page_table", "k_pool", "v_pool", "scores"):
            getattr(c, name).copy_(getattr(u, name))
        o.fill_(7)
        lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert int(c.error) == 0
        check_attend(u, True, o.cpu(), lse.cpu())
        ref, bound = weights64(u, lse.cpu(), True)
        assert ((c.scores.cpu().double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_as_many_sequences_as_there_may_be(kvc, dtype):
    """65,535 sequences of up to 40 tokens, a row each: append, attention, weights, eviction."""
    b, d, keep = 65535, 64, 20
    dt = DTYPES[dtype]
    g = torch.Generator(device=DEV).manual_seed(1)
    normal = lambda *s: torch.randn(s, generator=g, device=DEV).to(dt)
    k_pool, v_pool = normal(b * 3, 1, 16, d), normal(b * 3, 1, 16, d)
    table = torch.randperm(b * 3, generator=g, device=DEV).to(torch.int32).view(b, 3)
    lengths = (torch.arange(b, device=DEV) % 40).to(torch.int32)
    after = lengths.clone()
    scores, positions = torch.zeros(b, 1, 48, device=DEV), torch.arange(48, device=DEV).to(torch.int32).expand(b, 1, -1).contiguous()
    error = torch.zeros(1, dtype=torch.int32, device=DEV)
    batch = kvc.make_paged_batch(k_pool, v_pool, table, lengths, 1, d ** -0.5, next_positions=after, scores=scores,
                                 positions=positions, error=error)
    rows = torch.arange(b + 1, device=DEV).to(torch.int32)
    q, k, v = normal(b, 1, d), normal(b, 1, d), normal(b, 1, d)
    work = torch.empty(kvc.kvc_paged_workspace(batch, b, keep), dtype=torch.uint8, device=DEV)
    o, lse = torch.empty_like(q), torch.empty(b, 1, device=DEV)
    kvc.kvc_paged_append(batch, k, v, rows)
    kvc.kvc_paged_attend(batch, q, o, rows, work, lse=lse)
    kvc.kvc_paged_weights(batch, q, lse, rows, work)
    torch.cuda.synchronize()
    n = (torch.arange(b, device=DEV) % 40) + 1
    assert int(error) == 0 and torch.equal(lengths, n.to(torch.int32)) and torch.equal(after, lengths)
    own = lambda pool: pool[table.long(), 0].reshape(b, 48, d)
    at = torch.arange(b, device=DEV)
    assert torch.equal(own(k_pool)[at, n - 1], k[:, 0]) and torch.equal(own(v_pool)[at, n - 1], v[:, 0])
    there = torch.arange(48, device=DEV).view(1, -1) < n.view(-1, 1)
    keys, values, q64 = own(k_pool).double(), own(v_pool).double(), q.double()
    zero = torch.zeros((), dtype=torch.float64, device=DEV)
    x = torch.where(there, (keys * q64).sum(-1) * d ** -0.5, zero - math.inf)
    a = torch.where(there, (keys * q64).abs().sum(-1) * d ** -0.5, zero)
    w = torch.softmax(x, -1)
    # the bounds of attend64 and weights64
    u, half = 2.0 ** -24, torch.finfo(dt).eps / 2
    slack = 4 * (d + 2) * u * a.amax(-1, keepdim=True)
    e = torch.expm1(2 * slack) + 2.0 ** -21 + 96 * u
    ref, mass = (w.unsqueeze(-1) * values).sum(1), (w.unsqueeze(-1) * values.abs()).sum(1)
    bound = (2 * e + (half if dt != torch.float32 else 0)) * mass * 1.01 + half * ref.abs() * 1.01
    assert ((o[:, 0].double() - ref).abs() <= bound).all()
    assert ((lse.double() - torch.logsumexp(x, -1, keepdim=True)).abs() <=
            2 * slack + e + 4 * u * lse.double().abs() + 2.0 ** -21).all()
    y = lse.double()
    grow = torch.where(there, torch.exp(x - y), zero)
    slack = 4 * (d + 2) * u * a + 4 * u * (y.abs() + a)
    limit = grow * (torch.expm1(2 * slack) + 2.0 ** -21 + 6 * u) + 4 * u * grow
    assert ((scores[:, 0].double() - grow).abs() <= limit).all()
    # eviction: the kept tokens' scores, and every token with the key and value that it came with
    held, k_old = scores[:, 0].clone(), own(k_pool).clone()
    kvc.kvc_paged_evict(batch, keep, 2, 5, work)
    torch.cuda.synchronize()
    assert int(error) == 0 and torch.equal(lengths, n.clamp(max=keep).to(torch.int32))
    cut = (n > keep).nonzero().view(-1)
    pos = torch.arange(48, device=DEV).view(1, -1)
    key = torch.where((pos < 2) | (pos >= (n - 5).view(-1, 1)), torch.full_like(held, math.inf), held)
    key = torch.where(there, key, torch.full_like(held, -1.0))[cut]
    best = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :keep]
    kept = positions[cut, 0, :keep].long()
    assert torch.equal(kept.sort(1).values, best.sort(1).values)
    assert torch.equal(scores[cut, 0, :keep], held[cut].gather(1, kept))
    assert torch.equal(own(k_pool)[cut, :keep], k_old[cut].gather(1, kept.unsqueeze(-1).expand(-1, -1, d)))


@pytest.mark.parametrize("dtype,d,page", [("bf16", 64, 16), ("f32", 128, 32)])
def test_evict_many_heads(kvc, dtype, d, page):
    """So many heads that a CTA takes all of a head's moves, with room for many more tokens."""
    b, hkv, keep = 310, 8, 105
    t = Batch(rows=[1] * b, lengths=[keep + i for i in range(b)], hq=hkv, hkv=hkv, d=d, page=page, dtype=DTYPES[dtype],
              seed=3, stale=1.0, room=100)
    g = torch.Generator().manual_seed(4)
    t.scores = torch.randint(0, 50, t.scores.shape, generator=g).float()
    t.next_positions += 3
    c = copy.deepcopy(t).to(DEV)
    batch = c.handle(kvc)
    kvc.kvc_paged_evict(batch, keep, 4, 10, c.workspace(kvc, batch, keep))
    torch.cuda.synchronize()
    evict_sorted(t, keep, 4, 10)
    same_state(c, t, "many heads")
    assert int(c.error) == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_behind_the_last_sequence_change_nothing(kvc, dtype):
    """Rows of a padded batch hold NaN and infinities: every result is the same, bit for bit."""
    base = dict(rows=[3, 0, 150, 1], lengths=[40, 7, 333, 129], hq=4, hkv=2, d=64, prefix=50, room=160, behind=200)
    runs = []
    for value in (0.0, math.nan, math.inf):
        t = Batch(**base, dtype=DTYPES[dtype], seed=6)
        total = int(t.row_start[-1])
        t.q[total:] = value
        c = copy.deepcopy(t).to(DEV)
        batch = c.handle(kvc)
        work = c.workspace(kvc, batch, 30)
        k, v = (x.clone() for x in append_inputs(t))
        k[total:], v[total:] = value, value
        o, lse = torch.full(c.q.shape, 7.0, dtype=t.dtype, device=DEV), torch.full(c.q.shape[:2], 7.0, device=DEV)
        lse[total:] = value
        kvc.kvc_paged_append(batch, k.to(DEV), v.to(DEV), c.row_start)
        kvc.kvc_paged_attend(batch, c.q, o, c.row_start, work, lse=lse)
        kvc.kvc_paged_weights(batch, c.q, lse, c.row_start, work)
        kvc.kvc_paged_evict(batch, 30, 2, 5, work)
        torch.cuda.synchronize()
        assert int(c.error) == 0 and (o[total:] == 7).all()
        runs.append([x.cpu() for x in (o[:total], lse[:total], c.scores, c.positions, c.lengths,
                                       c.k_pool.view(torch.uint8), c.v_pool.view(torch.uint8))])
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)
