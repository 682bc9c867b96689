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
