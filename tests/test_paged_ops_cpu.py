"""Refusals of the paged-cache entry points (page planning, row append, dense chunk attention): bad
arguments come back with the documented status, before anything touches the device."""
import ctypes

import pytest
import torch

import sparse_mla_attention_fwd_gb300 as smla
from sparse_mla_attention_fwd_gb300 import _native
from sparse_mla_attention_fwd_gb300.native_build import build

FAKE = 1 << 30   # an aligned non-null "device" address; never dereferenced on error paths
STEP = 1 << 24   # buffers of the calls below lie this far apart
NULL, SHAPE, MISALIGNED, WORKSPACE = 1, 2, 3, 7


@pytest.fixture(scope="module")
def lib():
    build()
    return _native.load_library()


def plan(lib, **kw):
    names = ("seqlens", "new_lens", "table", "free", "start", "seqlens_k", "cu", "slots", "positions", "counts")
    a = {n: FAKE + i * STEP for i, n in enumerate(names)}
    a.update(n_req=4, n_free=100, n_tokens=64, max_blocks=8, page=64)
    a.update(kw)
    return lib.sparse_mla_plan_pages(*[a[n] for n in names], a["n_req"], a["n_free"], a["n_tokens"], a["max_blocks"],
                                     a["page"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_req=-1), SHAPE), (dict(n_free=-1), SHAPE), (dict(n_tokens=-1), SHAPE), (dict(n_tokens=1 << 31), SHAPE),
    (dict(max_blocks=0), SHAPE), (dict(page=0), SHAPE), (dict(max_blocks=1 << 20, page=1 << 12), SHAPE),
    (dict(seqlens=None), NULL), (dict(new_lens=None), NULL), (dict(table=None), NULL), (dict(free=None), NULL),
    (dict(seqlens_k=None), NULL), (dict(cu=None), NULL), (dict(slots=None), NULL), (dict(positions=None), NULL),
    (dict(counts=None), NULL), (dict(seqlens=FAKE + 2), MISALIGNED), (dict(counts=FAKE + 9 * STEP + 1), MISALIGNED),
    # outputs on top of inputs, or of one another
    (dict(seqlens_k=FAKE), SHAPE), (dict(start=FAKE + 9 * STEP + 4), SHAPE), (dict(positions=FAKE + 7 * STEP + 252), SHAPE),
    (dict(free=FAKE + 2 * STEP + 124), SHAPE),
])
def test_plan_refusals(lib, kw, code):
    assert plan(lib, **kw) == code


def append(lib, **kw):
    names = ("c", "k", "slots", "positions", "rope", "w", "q_pe", "q", "pool")
    a = {n: FAKE + i * STEP for i, n in enumerate(names)}
    a.update(cs=576, ks=576, max_pos=100, eps=1e-6, qt=24 * 64, qh=64, h=24, rows=128, d=576, n=5)
    a.update(kw)
    return lib.sparse_mla_append_kv(a["c"], a["cs"], a["k"], a["ks"], a["slots"], a["positions"], a["rope"], a["max_pos"],
                                    a["w"], ctypes.c_float(a["eps"]), a["q_pe"], a["qt"], a["qh"], a["q"], a["h"],
                                    a["pool"], a["rows"], a["d"], a["n"], None)


NO_ROPE = dict(d=512, k=None, rope=None, q_pe=None, q=None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=640), SHAPE), (dict(n=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(max_pos=0), SHAPE), (dict(h=0), SHAPE), (dict(h=1025), SHAPE),
    (dict(cs=-8), SHAPE), (dict(NO_ROPE, rope=FAKE), SHAPE),
    (dict(c=None), NULL), (dict(k=None), NULL), (dict(slots=None), NULL), (dict(pool=None), NULL),
    (dict(positions=None), NULL), (dict(q=None), NULL), (dict(q_pe=None), NULL), (dict(rope=None), NULL),
    (dict(NO_ROPE, k=FAKE + STEP), NULL),
    (dict(cs=577), MISALIGNED), (dict(c=FAKE + 8), MISALIGNED), (dict(ks=575), MISALIGNED), (dict(k=FAKE + STEP + 2), MISALIGNED),
    (dict(qt=1540), MISALIGNED), (dict(qh=68), MISALIGNED), (dict(pool=FAKE + 8 * STEP + 8), MISALIGNED),
    (dict(rope=FAKE + 4 * STEP + 4), MISALIGNED), (dict(w=FAKE + 5 * STEP + 2), MISALIGNED),
    (dict(pool=FAKE + 4096), SHAPE), (dict(pool=FAKE + STEP), SHAPE),   # rows on top of the inputs
])
def test_append_refusals(lib, kw, code):
    assert append(lib, **kw) == code


Q, Q_PE = FAKE + 7 * STEP, FAKE + 6 * STEP


@pytest.mark.parametrize("kw", [
    dict(q_pe=Q), dict(q_pe=Q + 1024 - 16, qt=24 * 576, qh=576), dict(q_pe=Q + 1024, qt=24 * 576, qh=64),   # beside its place
    dict(q_pe=Q + 1024, qt=64, qh=576), dict(q_pe=Q + 5 * 24 * 1152 - 16), dict(q_pe=Q, qt=0, qh=0),
    dict(q=FAKE), dict(q=FAKE + STEP), dict(q=FAKE + 8 * STEP), dict(q=FAKE + 8 * STEP + 1152 * 127),
    dict(q_pe=FAKE + 8 * STEP), dict(pool=Q_PE + 4096),
])
def test_append_refuses_overlapping_queries(lib, kw):
    assert append(lib, **kw) == SHAPE


def test_append_of_nothing(lib):
    assert append(lib, n=0, c=None, k=None, slots=None, positions=None) == 0
    assert append(lib, n=0, c=None, slots=None, **NO_ROPE) == 0


def chunk(lib, **kw):
    a = dict(q=FAKE, pool=FAKE, rows=4096, table=FAKE, max_blocks=64, page=64, cu=FAKE, seqlens=FAKE, n_req=3, causal=1,
             sink=None, scale=0.04, d_v=512, out=FAKE, lse=FAKE, mx=FAKE, n_tok=9, h=128, d=576, ws=FAKE, nbytes=1 << 40)
    a.update(kw)
    return lib.sparse_mla_chunk_fwd_paged(a["q"], a["pool"], a["rows"], a["table"], a["max_blocks"], a["page"], a["cu"],
                                          a["seqlens"], a["n_req"], a["causal"], a["sink"], ctypes.c_float(a["scale"]),
                                          a["d_v"], a["out"], a["lse"], a["mx"], a["n_tok"], a["h"], a["d"], a["ws"],
                                          a["nbytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(h=0), SHAPE), (dict(h=1025), SHAPE), (dict(d=640), SHAPE), (dict(d_v=256), SHAPE), (dict(n_tok=-1), SHAPE),
    (dict(n_req=-1), SHAPE), (dict(n_tok=1 << 24), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(rows=0), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(page=0), SHAPE), (dict(max_blocks=0), SHAPE),
    (dict(max_blocks=1 << 16, page=1 << 15), SHAPE),
    (dict(q=None), NULL), (dict(pool=None), NULL), (dict(table=None), NULL), (dict(cu=None), NULL),
    (dict(seqlens=None), NULL), (dict(out=None), NULL), (dict(lse=None), NULL), (dict(mx=None), NULL),
    (dict(q=FAKE + 8), MISALIGNED), (dict(pool=FAKE + 2), MISALIGNED), (dict(out=FAKE + 4), MISALIGNED),
    (dict(table=FAKE + 2), MISALIGNED), (dict(sink=FAKE + 1), MISALIGNED),
])
def test_chunk_refusals(lib, kw, code):
    assert chunk(lib, **kw) == code


def test_chunk_of_nothing(lib):
    nothing = dict(q=None, pool=None, table=None, cu=None, seqlens=None, out=None, lse=None, mx=None, ws=None, nbytes=0)
    assert chunk(lib, n_tok=0, **nothing) == 0
    assert chunk(lib, n_req=0, **nothing) == 0


def test_wrappers_reject_wrong_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    b = torch.zeros((4, 1, 576), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        smla.sparse_mla_plan_pages(i, i, i.view(2, 2), i, 4)
    with pytest.raises(TypeError):
        smla.sparse_mla_plan_pages(i.long(), i, i.view(2, 2), i, 4)
    with pytest.raises(ValueError):
        smla.sparse_mla_append_kv(b[:, 0, :512], b[:, 0, 512:], i, b)
    with pytest.raises(TypeError):
        smla.sparse_mla_append_kv(b[:, 0, :512], b[:, 0, 512:], i, b.float())
    with pytest.raises(ValueError):
        smla.sparse_mla_chunk_fwd_paged(b, b, i.view(2, 2), i, i)
    with pytest.raises(TypeError):
        smla.sparse_mla_chunk_fwd_paged(b.float(), b, i.view(2, 2), i, i)


def test_counted_append_refusals(lib):
    def call(past, **kw):
        a = dict(c=FAKE, k=FAKE + STEP, pool=FAKE + 8 * STEP, n=5)
        a.update(kw)
        return lib.sparse_mla_append_kv_counted(
            a["c"], 576, a["k"], 576, FAKE + 2 * STEP, FAKE + 3 * STEP, FAKE + 4 * STEP, 100, None, ctypes.c_float(1e-6),
            FAKE + 6 * STEP, 24 * 64, 64, FAKE + 7 * STEP, 24, a["pool"], 128, 576, a["n"], past, None)

    free = FAKE + 9 * STEP
    assert call(None) == NULL
    assert call(free + 2) == MISALIGNED
    assert call(FAKE + 8 * STEP + 128 * 1152 - 4) == SHAPE     # the cache's last bytes
    assert call(FAKE + 7 * STEP + 1024) == SHAPE               # the queries'
    assert call(FAKE + 2 * STEP + 16) == SHAPE and call(FAKE + 3 * STEP) == SHAPE   # slots, positions
    assert call(free, c=None) == NULL and call(free, pool=FAKE + 4096) == SHAPE
    assert call(free, n=0) == 0


def test_strides_of_one_token_or_head_are_not_looked_at(lib):
    """With the strides accepted, each call comes to the overlap check, which refuses it."""
    over = dict(pool=FAKE)
    assert append(lib, n=1, cs=1, ks=1, qt=-3, qh=64, **over) == SHAPE
    assert append(lib, h=1, qh=1, qt=64, **over) == SHAPE
    assert append(lib, n=1, h=1, cs=5, ks=5, qt=5, qh=5, **over) == SHAPE
    assert append(lib, n=2, cs=5, **over) == MISALIGNED and append(lib, h=2, qh=5, **over) == MISALIGNED


APART = {n: FAKE + (i << 28) for i, n in enumerate(("q", "pool", "table", "cu", "seqlens", "sink", "out", "lse", "mx", "ws"))}
SIZES = dict(q=9 * 128 * 1152, pool=4096 * 1152, table=3 * 64 * 4, cu=16, seqlens=12, sink=512, out=9 * 128 * 1024, lse=9 * 128 * 4,
             mx=9 * 128 * 4, ws=160 * 128 * 2048)


@pytest.mark.parametrize("written,other", [(a, b) for a in ("out", "lse", "mx", "ws") for b in APART if a != b])
def test_chunk_refuses_overlapping_buffers(lib, written, other):
    size = SIZES[other] - SIZES[other] % 256 or 256
    at = [APART[other], APART[other] + size - 256]      # on its first bytes, and on its last
    for a in at:
        assert chunk(lib, **dict(APART, **{written: a})) == SHAPE


def test_wait_selftest_refuses_limits_out_of_range(lib):
    for limit in (0, 2_000_000_001, 2 ** 64 - 1):
        assert lib.sparse_mla_chunk_selftest_wait_timeout(limit, None) == SHAPE


@pytest.mark.parametrize("written", ["pool", "q"])
@pytest.mark.parametrize("read,size", [("slots", 20), ("positions", 20), ("rope", 100 * 256), ("w", 1024)])
def test_append_refuses_to_write_on_what_it_reads(lib, written, read, size):
    at = {"pool": FAKE + 8 * STEP, "q": FAKE + 7 * STEP}[written]
    end = at + {"pool": 128 * 1152, "q": 5 * 24 * 1152}[written]
    for a in (at, end - 16, at - (size - 1) // 16 * 16):      # its first bytes, its last, and from below
        assert append(lib, **{read: a}) == SHAPE
