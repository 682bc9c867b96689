"""The paged-batch operators at the ends of their ranges: terms and scores that overflow, batches whose
rows are dealt out unevenly, and the forms that only large or full sequences take."""
import copy
import math

import pytest
import torch

from paged_util import Batch, append_ref, weights64
from test_gpu_paged import DEV, DTYPES, same_state

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
