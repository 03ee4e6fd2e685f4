"""Refusals of a speculative step's entry points (tree planning, tree attention, verification, commit): bad arguments come
back with the documented status, before anything touches the device."""
import ctypes

import pytest
import torch

import sparse_mla_attention_fwd_gb300 as smla
from sparse_mla_attention_fwd_gb300 import _native
from sparse_mla_attention_fwd_gb300.native_build import build

FAKE = 1 << 30   # an aligned non-null "device" address; never dereferenced on error paths
STEP = 1 << 28   # buffers of the calls below lie this far apart
NULL, SHAPE, MISALIGNED, WORKSPACE = 1, 2, 3, 7


@pytest.fixture(scope="module")
def lib():
    build()
    return _native.load_library()


def apart(*names):
    return {n: FAKE + i * STEP for i, n in enumerate(names)}


# ------------------------------------------------------------------------------ tree planning
PLAN = apart("parents", "cu", "seqlens_k", "mask", "positions")


def plan(lib, **kw):
    a = dict(PLAN, n_req=4, n_tok=64, words=2)
    a.update(kw)
    return lib.sparse_mla_plan_tree(*[a[n] for n in PLAN], a["n_req"], a["n_tok"], a["words"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_req=-1), SHAPE), (dict(n_tok=-1), SHAPE), (dict(n_req=1 << 31), SHAPE), (dict(n_tok=1 + (1 << 30)), SHAPE),
    (dict(words=0), SHAPE), (dict(words=1025), SHAPE),
    *[({n: None}, NULL) for n in PLAN], *[({n: PLAN[n] + 2}, MISALIGNED) for n in PLAN],
    (dict(mask=FAKE), SHAPE), (dict(mask=FAKE + STEP + 16), SHAPE), (dict(positions=FAKE + 2 * STEP + 12), SHAPE),
    (dict(positions=PLAN["mask"] + 64 * 8 - 4), SHAPE), (dict(mask=FAKE - 64 * 8 + 4), SHAPE),
])
def test_plan_refusals(lib, kw, code):
    assert plan(lib, **kw) == code


def test_plan_of_nothing(lib):
    assert plan(lib, n_tok=0, **{n: None for n in PLAN}) == 0


# ----------------------------------------------------------------------------- tree attention
TREE = apart("q", "pool", "table", "cu", "seqlens", "mask", "sink", "out", "lse", "mx", "ws")
SIZES = dict(q=9 * 128 * 1152, pool=4096 * 1152, table=3 * 64 * 4, cu=16, seqlens=12, mask=9 * 2 * 4, sink=512,
             out=9 * 128 * 1024, lse=9 * 128 * 4, mx=9 * 128 * 4, ws=160 * 128 * 2048)


def tree(lib, **kw):
    a = dict(TREE, rows=4096, max_blocks=64, page=64, n_req=3, words=2, scale=0.04, d_v=512, n_tok=9, h=128, d=576,
             nbytes=1 << 40)
    a.update(kw)
    return lib.sparse_mla_tree_fwd_paged(a["q"], a["pool"], a["rows"], a["table"], a["max_blocks"], a["page"], a["cu"],
                                         a["seqlens"], a["n_req"], a["mask"], a["words"], a["sink"], ctypes.c_float(a["scale"]),
                                         a["d_v"], a["out"], a["lse"], a["mx"], a["n_tok"], a["h"], a["d"], a["ws"],
                                         a["nbytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(h=0), SHAPE), (dict(h=1025), SHAPE), (dict(d=640), SHAPE), (dict(d_v=256), SHAPE), (dict(n_tok=-1), SHAPE),
    (dict(n_req=-1), SHAPE), (dict(n_tok=1 << 24), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(rows=0), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(page=0), SHAPE), (dict(max_blocks=0), SHAPE),
    (dict(max_blocks=1 << 16, page=1 << 15), SHAPE), (dict(words=0), SHAPE), (dict(words=1025), SHAPE),
    *[({n: None}, NULL) for n in TREE if n not in ("sink", "ws")], (dict(ws=None), WORKSPACE), (dict(nbytes=4096), WORKSPACE),
    *[({n: TREE[n] + 2}, MISALIGNED) for n in TREE], (dict(ws=TREE["ws"] + 128), MISALIGNED),
])
def test_tree_refusals(lib, kw, code):
    assert tree(lib, **kw) == code


@pytest.mark.parametrize("written,other", [(a, b) for a in ("out", "lse", "mx", "ws") for b in TREE if a != b])
def test_tree_refuses_overlapping_buffers(lib, written, other):
    size = SIZES[other] - SIZES[other] % 256 or 256
    for at in (TREE[other], TREE[other] + size - 256):      # on its first bytes, and on its last
        assert tree(lib, **{written: at}) == SHAPE


def test_tree_of_nothing(lib):
    nothing = {n: None for n in TREE}
    assert tree(lib, n_tok=0, nbytes=0, **nothing) == 0
    assert tree(lib, n_req=0, nbytes=0, **nothing) == 0


# ------------------------------------------------------------------------------- verification
VERIFY = apart("target", "draft", "tokens", "parents", "cu", "accept", "sample", "keep", "out", "n_keep")
V_SIZES = dict(target=(11 * 1040 + 1001) * 4, draft=(11 * 1001 + 1001) * 4, tokens=48, parents=48, cu=16, accept=48, sample=12,
               keep=3 * 5 * 4, out=3 * 5 * 4, n_keep=12)


def verify(lib, **kw):
    a = dict(VERIFY, ts=1040, ds=1001, n_req=3, n_tok=12, vocab=1001, max_keep=5)
    a.update(kw)
    return lib.sparse_mla_verify_tree(a["target"], a["ts"], a["draft"], a["ds"], a["tokens"], a["parents"], a["cu"], a["accept"],
                                      a["sample"], a["keep"], a["out"], a["n_keep"], a["n_req"], a["n_tok"], a["vocab"],
                                      a["max_keep"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_req=-1), SHAPE), (dict(n_tok=-1), SHAPE), (dict(n_req=1 << 31), SHAPE), (dict(n_tok=1 << 31), SHAPE),
    (dict(vocab=0), SHAPE), (dict(vocab=(1 << 30) + 1, ts=1 << 31, ds=1 << 31), SHAPE), (dict(max_keep=0), SHAPE), (dict(n_req=1 << 20, max_keep=1 << 11), SHAPE),
    (dict(ts=1000), SHAPE), (dict(ds=1000), SHAPE), (dict(ts=-1040), SHAPE), (dict(ts=1 << 61), SHAPE), (dict(ds=1 << 61), SHAPE),
    *[({n: None}, NULL) for n in VERIFY if n != "draft"], *[({n: VERIFY[n] + 2}, MISALIGNED) for n in VERIFY],
])
def test_verify_refusals(lib, kw, code):
    assert verify(lib, **kw) == code


@pytest.mark.parametrize("written,other", [(a, b) for a in ("keep", "out", "n_keep") for b in VERIFY if a != b])
def test_verify_refuses_overlapping_buffers(lib, written, other):
    for at in (VERIFY[other], VERIFY[other] + V_SIZES[other] - 4, VERIFY[other] - V_SIZES[written] + 4):
        assert verify(lib, **{written: at}) == SHAPE


def test_verify_of_nothing(lib):
    assert verify(lib, n_req=0, **{n: None for n in VERIFY}) == 0
    # the stride of a single row is not looked at: the call comes to the overlap check, which refuses it
    assert verify(lib, n_tok=1, ts=3, ds=-2, keep=VERIFY["out"]) == SHAPE


# ------------------------------------------------------------------------------------- commit
COMMIT = apart("keep", "n_keep", "cu", "seqlens_k", "table", "pool", "free", "start", "seqlens", "counts")
C_SIZES = dict(keep=3 * 5 * 4, n_keep=12, cu=16, seqlens_k=12, table=3 * 8 * 4, pool=(64 * 576 + 40000) * 2, free=400, start=4,
               seqlens=12, counts=12)


def commit(lib, **kw):
    a = dict(COMMIT, max_keep=5, max_blocks=8, page=16, n_req=3, layers=2, stride=40000, rows=64, d=576, n_free=100)
    a.update(kw)
    return lib.sparse_mla_commit_tree(a["keep"], a["n_keep"], a["max_keep"], a["cu"], a["seqlens_k"], a["table"],
                                      a["max_blocks"], a["page"], a["n_req"], a["pool"], a["layers"], a["stride"], a["rows"],
                                      a["d"], a["free"], a["n_free"], a["start"], a["seqlens"], a["counts"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_req=-1), SHAPE), (dict(n_req=1 << 31), SHAPE), (dict(max_keep=0), SHAPE), (dict(n_req=1 << 20, max_keep=1 << 11), SHAPE),
    (dict(max_blocks=0), SHAPE), (dict(page=0), SHAPE), (dict(max_blocks=1 << 16, page=1 << 15), SHAPE), (dict(layers=-1), SHAPE),
    (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(n_free=-1), SHAPE), (dict(n_free=1 << 31), SHAPE), (dict(d=640), SHAPE),
    (dict(stride=64 * 576 - 8), SHAPE), (dict(stride=-40000), SHAPE), (dict(stride=1 << 61), SHAPE), (dict(stride=40004), MISALIGNED),
    *[({n: None}, NULL) for n in COMMIT if n not in ("free", "start")], *[({n: COMMIT[n] + 2}, MISALIGNED) for n in COMMIT],
    (dict(pool=COMMIT["pool"] + 8), MISALIGNED), (dict(free=None, n_free=0, seqlens=None), NULL),
])
def test_commit_refusals(lib, kw, code):
    assert commit(lib, **kw) == code


@pytest.mark.parametrize("written,other", [(a, b) for a in ("pool", "free", "seqlens", "counts") for b in COMMIT if a != b])
def test_commit_refuses_overlapping_buffers(lib, written, other):
    size = C_SIZES[other] - C_SIZES[other] % 16 or 16
    for at in (COMMIT[other], COMMIT[other] + size - 16):
        assert commit(lib, **{written: at}) == SHAPE


def test_commit_does_not_look_at_a_single_layers_stride(lib):
    assert commit(lib, layers=1, stride=-7, seqlens=COMMIT["counts"]) == SHAPE     # the overlap is what is refused
    assert commit(lib, layers=1, stride=7, counts=None) == NULL


def test_wrappers_reject_wrong_tensors():
    i, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 8)
    b = torch.zeros((4, 1, 576), dtype=torch.bfloat16)
    for call, args in ((smla.sparse_mla_plan_tree, (i, i, i, 1)), (smla.sparse_mla_tree_fwd_paged, (b, b, i.view(2, 2), i, i, i.view(4, 1))),
                       (smla.sparse_mla_verify_tree, (f, i, i, i, f[:, 0].contiguous(), f[:, 0].contiguous(), 2)),
                       (smla.sparse_mla_commit_tree, (i.view(2, 2), i, i, i, i.view(2, 2), b))):
        with pytest.raises(ValueError):       # not on a GPU
            call(*args)
    with pytest.raises(TypeError):
        smla.sparse_mla_plan_tree(i.long(), i, i, 1)
    with pytest.raises(TypeError):
        smla.sparse_mla_tree_fwd_paged(b.float(), b, i.view(2, 2), i, i, i.view(4, 1))
    with pytest.raises(TypeError):
        smla.sparse_mla_verify_tree(f, i.long(), i, i, f[0], f[0], 2)
    with pytest.raises(TypeError):
        smla.sparse_mla_commit_tree([[0]], i, i, i, i.view(2, 2), b)
