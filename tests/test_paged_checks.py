"""The paged-batch entry points' checks, none of which needs a GPU: the struct's layout, every
rule of the C entry points with fake addresses, and what the binding refuses."""
import ctypes
import os
import subprocess
import tempfile
import types

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

OK, ARG, CUDA, UNSUPPORTED = 0, 1, 3, 8


def test_batch_layout_matches_header():
    import transformer_kv_cache_b200 as kvc
    names = [n for n, _ in kvc.kvc_paged_batch._fields_]
    prog = "#include <stdio.h>\n#include <stddef.h>\n#include \"kvc.h\"\nint main(void) {\n" \
           "  printf(\"%zu\", sizeof(kvc_paged_batch));\n" + \
           "".join(f"  printf(\" %zu\", offsetof(kvc_paged_batch, {n}));\n" for n in names) + "  return 0;\n}\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write(prog)
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True).stdout.split()]
    B = kvc.kvc_paged_batch
    assert got == [ctypes.sizeof(B)] + [getattr(B, n).offset for n in names]


BATCH = dict(dtype=1, num_seqs=3, num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=16, max_pages=40,
             prefix_tokens=100, pool_pages=500, k_pool=0x10000, v_pool=0x20000, page_table=0x30000, lengths=0x40000,
             prefix_pages=0x50000, next_positions=0x60000, scores=0x70000, positions=0x80000, error=0x90000,
             softmax_scale=0.125, reserved=0)
CALLS = {
    "append": dict(k=0x100000, v=0x110000, k_stride=128, v_stride=128, rows=5, row_start=0x120000),
    "attend": dict(q=0x100000, stride=512, o=0x110000, lse=0x130000, rows=5, row_start=0x120000, causal=1,
                   work=0x140000, bytes=1 << 40),
    "weights": dict(q=0x100000, stride=512, lse=0x130000, rows=5, row_start=0x120000, causal=1, work=0x140000,
                    bytes=1 << 40),
    "evict": dict(keep=64, sinks=4, recent=16, work=0x140000, bytes=1 << 40),
    "workspace": dict(rows=5, keep=64),
}


def call(name, batch=None, **over):
    import transformer_kv_cache_b200 as kvc
    b = kvc.kvc_paged_batch()
    for k, v in {**BATCH, **(batch or {})}.items():
        setattr(b, k, v)
    a = {**CALLS[name], **over}
    r, L = ctypes.byref(b), kvc._lib
    if name == "append":
        return L.kvc_paged_append(r, a["k"], a["v"], a["k_stride"], a["v_stride"], a["rows"], a["row_start"], None)
    if name == "attend":
        return L.kvc_paged_attend(r, a["q"], a["stride"], a["o"], a["lse"], a["rows"], a["row_start"], a["causal"],
                                  a["work"], a["bytes"], None)
    if name == "weights":
        return L.kvc_paged_weights(r, a["q"], a["stride"], a["lse"], a["rows"], a["row_start"], a["causal"], a["work"],
                                   a["bytes"], None)
    if name == "evict":
        return L.kvc_paged_evict(r, a["keep"], a["sinks"], a["recent"], a["work"], a["bytes"], None)
    out = ctypes.c_int64(0)
    return L.kvc_paged_workspace(r, a["rows"], a["keep"], ctypes.byref(out))


# one rule of the batch at a time: every call refuses it
BATCH_RULES = [
    (dict(dtype=2), "FP8 storage"),
    (dict(dtype=-1), "no type"),
    (dict(num_seqs=0), "no sequences"),
    (dict(num_seqs=65536), "too many sequences"),
    (dict(num_kv_heads=0), "no KV heads"),
    (dict(num_q_heads=0), "no query heads"),
    (dict(num_q_heads=7), "query heads no multiple of KV heads"),
    (dict(num_q_heads=130), "a group of more than 64"),
    (dict(head_dim=32), "32 dims"),
    (dict(head_dim=96), "96 dims"),
    (dict(page_size=8), "pages of 8"),
    (dict(page_size=48), "a page size that is no power of two"),
    (dict(page_size=512), "pages of 512"),
    (dict(max_pages=0), "no pages to a sequence"),
    (dict(max_pages=(1 << 26) + 1), "more slots than an index holds"),
    (dict(prefix_tokens=-1), "a negative prefix"),
    (dict(prefix_pages=None), "a prefix without pages"),
    (dict(pool_pages=0), "an empty pool"),
    (dict(pool_pages=1 << 26), "more pool rows than an index holds"),
    (dict(k_pool=None), "no K pool"),
    (dict(v_pool=None), "no V pool"),
    (dict(page_table=None), "no page table"),
    (dict(lengths=None), "no lengths"),
    (dict(k_pool=0x10008), "K pool not 16-byte aligned"),
    (dict(v_pool=0x20002), "V pool not 16-byte aligned"),
    (dict(scores=0x70004), "scores not 16-byte aligned"),
    (dict(positions=0x80008), "positions not 16-byte aligned"),
    (dict(softmax_scale=0.0), "scale not positive"),
    (dict(softmax_scale=float("nan")), "scale NaN"),
    (dict(softmax_scale=float("inf")), "scale infinite"),
    (dict(reserved=1), "reserved word set"),
]


@pytest.fixture
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("fake device addresses: host checks only, on a host without a GPU")


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("change,why", BATCH_RULES, ids=[r[1] for r in BATCH_RULES])
def test_batch_rule_refused_by_every_call(no_gpu, name, change, why):
    assert call(name) == CUDA, "the base call passes the host checks and stops at the first CUDA call"
    assert call(name, batch=change) == ARG, why


CALL_RULES = [
    ("append", {}, dict(k=None), "no K"),
    ("append", {}, dict(v=None), "no V"),
    ("append", {}, dict(k=0x100008), "K not aligned"),
    ("append", {}, dict(k_stride=120), "rows that overlap"),
    ("append", {}, dict(v_stride=132), "a stride that leaves rows unaligned"),
    ("append", {}, dict(rows=-1), "negative rows"),
    ("append", {}, dict(row_start=None), "no row starts"),
    ("append", dict(next_positions=None), {}, "positions without the next ones"),
    ("attend", {}, dict(q=None), "no Q"),
    ("attend", {}, dict(o=None), "no O"),
    ("attend", {}, dict(o=0x110008), "O not aligned"),
    ("attend", {}, dict(stride=504), "query rows that overlap"),
    ("attend", {}, dict(rows=-1), "negative rows"),
    ("attend", {}, dict(row_start=None), "no row starts"),
    ("attend", {}, dict(causal=2), "no truth value"),
    ("attend", {}, dict(work=None), "no workspace"),
    ("attend", {}, dict(work=0x140004), "workspace not aligned"),
    ("attend", {}, dict(rows=2 ** 30), "more row-heads than a merge holds"),
    ("weights", dict(scores=None), {}, "no scores"),
    ("weights", {}, dict(q=None), "no Q"),
    ("weights", {}, dict(lse=None), "no log-sum-exp"),
    ("weights", {}, dict(stride=516), "a stride that leaves rows unaligned"),
    ("weights", {}, dict(row_start=None), "no row starts"),
    ("weights", {}, dict(work=None), "no workspace"),
    ("weights", {}, dict(causal=-1), "no truth value"),
    ("evict", dict(scores=None), {}, "no scores"),
    ("evict", dict(positions=None), {}, "no positions"),
    ("evict", dict(next_positions=None), {}, "no next positions"),
    ("evict", {}, dict(keep=0), "nothing kept"),
    ("evict", {}, dict(sinks=-1), "negative sinks"),
    ("evict", {}, dict(recent=-1), "negative recent tokens"),
    ("evict", {}, dict(sinks=40, recent=25), "more protected than kept"),
    ("evict", {}, dict(work=None), "no workspace"),
    ("evict", {}, dict(bytes=64), "workspace too small"),
    ("workspace", {}, dict(rows=-1), "negative rows"),
    ("workspace", {}, dict(keep=-1), "negative keep"),
]


@pytest.mark.parametrize("name,batch,change,why", CALL_RULES, ids=[f"{r[0]}: {r[3]}" for r in CALL_RULES])
def test_call_rule_refused(no_gpu, name, batch, change, why):
    assert call(name, batch=batch, **change) == ARG, why


def test_calls_with_nothing_to_do_succeed(no_gpu):
    for name in ("append", "attend", "weights"):
        assert call(name, rows=0) == OK
    assert call("attend", rows=0, q=None, o=None) == OK
    assert call("evict", keep=40 * 16) == OK                  # no sequence can hold more
    assert call("evict", batch=dict(max_pages=1 << 15)) == UNSUPPORTED


def test_binding_refuses_host_buffers_and_wrong_tensors():
    import transformer_kv_cache_b200 as kvc
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(TypeError):
        kvc.make_paged_batch(pool, pool, i32(1, 4), i32(1), 2, 0.125)
    cpu = torch.device("cpu")
    # the checks of single tensors, on a stand-in for a batch
    x = torch.zeros(3, 4, 64)
    with pytest.raises(TypeError):                            # another type, and a host buffer
        kvc._packed("x", x, cpu, torch.bfloat16, x.shape)
    batch = types.SimpleNamespace(_device=cpu, _dtype=torch.float32, _dim=64)
    assert kvc._paged_rows(batch, "q", x, 4) == (x.data_ptr(), 256, 3)
    fused = torch.zeros(3, 12, 64)
    assert kvc._paged_rows(batch, "q", fused[:, 4:8], 4)[1] == 768
    for bad in (x[:, :3], x[:, :, :32], x.transpose(0, 1), fused[:, ::3], x[0]):
        with pytest.raises(ValueError):
            kvc._paged_rows(batch, "q", bad, 4)


def test_binding_refuses_numbers_past_32_bits():
    """ctypes would keep their lower 32 bits: 2^32 + 64 tokens to keep would be 64."""
    import transformer_kv_cache_b200 as kvc
    for bad in (2 ** 31, 2 ** 32 + 64, -2 ** 31 - 1):
        for name in ("keep", "sinks", "recent"):
            with pytest.raises(ValueError, match=name):
                kvc.kvc_paged_evict(None, **{**dict(keep=64, sinks=4, recent=16), name: bad}, workspace=None)
        for name in ("rows", "keep"):
            with pytest.raises(ValueError, match=name):
                kvc.kvc_paged_workspace(None, **{**dict(rows=5, keep=64), name: bad})
    kvc._int32(a=-2 ** 31, b=2 ** 31 - 1)


@pytest.mark.parametrize("name", CALLS)
def test_lengths_as_next_positions_refused(no_gpu, name):
    """An append grows both by its rows: in one array it would add them twice."""
    assert call(name, batch=dict(next_positions=BATCH["lengths"])) == ARG
