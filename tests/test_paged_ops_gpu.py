"""GPU tests of the paged-cache operators: page planning, row append, dense chunk attention, and a
serving step of the three together.

References are plain loops (planning, whole numbers: equal) or 64-bit torch on the same inputs.
Tolerances count roundings: u = 2^-8 for one rounding to bf16, 2^-24 for fp32."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import sparse_mla_attention_fwd_gb300 as smla

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U16, U32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(autouse=True)
def device_status():
    yield
    torch.cuda.synchronize()
    assert smla.sparse_mla_device_status() == 0


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


# ------------------------------------------------------------------------------ page planning
def plan_loops(old, new, table, free, n_tokens, page, start):
    table, n_free = table.copy(), len(free)
    width = table.shape[1]
    cu, length, slots, positions = [0], [], [-1] * n_tokens, [-1] * n_tokens
    at = max(start, 0)
    missing = 0
    for b, (o, m) in enumerate(zip(old, new)):
        o, m = max(o, 0), min(max(m, 0), n_tokens - cu[-1])
        for col in range(min(-(-o // page), width), min(-(-(o + m) // page), width)):
            table[b, col] = free[at] if at < n_free else -1
            missing += at >= n_free
            at += at < n_free
        for i in range(m):
            pos = o + i
            positions[cu[-1] + i] = pos
            if pos // page < width and table[b, pos // page] >= 0:
                slots[cu[-1] + i] = table[b, pos // page] * page + pos % page
        cu.append(cu[-1] + m)
        length.append(o + m)
    return length, cu, slots, positions, [cu[-1], at, missing], table


def plan_case(seed, n_req, page, old_max, new_max, width, n_free, pad=0, start=None, zeros=0.2, cut=0):
    rng = np.random.default_rng(seed)
    old = rng.integers(0, old_max + 1, n_req)
    new = rng.integers(0, new_max + 1, n_req) * (rng.random(n_req) >= zeros)
    table = rng.permutation(n_req * width).astype(np.int32).reshape(n_req, width)
    table[np.arange(width)[None, :] >= -(-old[:, None] // page)] = -1
    table[rng.random(table.shape) < 0.05] = -1
    free = 100000 + rng.permutation(n_free).astype(np.int32)
    return old, new, table, free, max(0, int(new.sum()) + pad - cut), page, start


@pytest.mark.parametrize("kw", [
    dict(n_req=0, page=64, old_max=1, new_max=1, width=3, n_free=4, pad=5),
    dict(n_req=1, page=64, old_max=500, new_max=1, width=9, n_free=4, zeros=0),
    dict(n_req=8, page=64, old_max=4000, new_max=1, width=64, n_free=20, start=3),
    dict(n_req=255, page=16, old_max=300, new_max=40, width=25, n_free=1000, pad=13),
    dict(n_req=256, page=1, old_max=30, new_max=9, width=64, n_free=3000, start=0),
    dict(n_req=257, page=7, old_max=100, new_max=100, width=40, n_free=9000, pad=1),
    dict(n_req=1000, page=100, old_max=2000, new_max=60, width=23, n_free=1000),
    dict(n_req=3, page=64, old_max=100, new_max=40000, width=700, n_free=2000, zeros=0),
    dict(n_req=40, page=16, old_max=100, new_max=50, width=25, n_free=30),              # too few pages
    dict(n_req=40, page=16, old_max=100, new_max=50, width=25, n_free=30, start=77),    # none
    dict(n_req=40, page=16, old_max=100, new_max=50, width=25, n_free=0),
    dict(n_req=40, page=16, old_max=400, new_max=300, width=20, n_free=900),            # past the table
    dict(n_req=300, page=16, old_max=100, new_max=50, width=25, n_free=900, cut=3000),  # more tokens than room
    dict(n_req=300, page=16, old_max=100, new_max=0, width=25, n_free=900, pad=2),
    dict(n_req=5, page=16, old_max=100, new_max=9, width=25, n_free=900, start=-4),
])
@pytest.mark.parametrize("seed", [0, 1])
def test_plan_against_loops(kw, seed):
    old, new, table, free, n_tokens, page, start = plan_case(seed, **kw)
    want = plan_loops(old, new, table, free, n_tokens, page, start or 0)
    args = (i32(old), i32(new), i32(table), i32(free), n_tokens)
    for _ in range(2):   # a second call on the same inputs gives the same
        got = smla.sparse_mla_plan_pages(*args, page_block=page, free_start=None if start is None else i32([start]))
        for g, w, name in zip(got, want, ("seqlens_k", "cu_seqlens_q", "slots", "positions", "counts")):
            assert np.array_equal(g.cpu().numpy(), np.asarray(w, dtype=np.int32)), name
        assert np.array_equal(args[2].cpu().numpy(), want[5])


def test_plan_takes_negative_lengths_as_zero():
    got = smla.sparse_mla_plan_pages(i32([-5, 3]), i32([2, -7]), i32([[-1, -1], [4, -1]]), i32([9, 8]), 4, page_block=4)
    assert [g.tolist() for g in got] == [[2, 3], [0, 2, 2], [36, 37, -1, -1], [0, 1, -1, -1], [2, 1, 0]]


def test_plan_chains_steps_through_counts():
    """Ten steps without the host looking: counts of one step are the next one's free_start."""
    rng = np.random.default_rng(5)
    n_req, page, width = 17, 8, 40
    old, table = np.zeros(n_req, dtype=np.int64), np.full((n_req, width), -1, dtype=np.int32)
    free = rng.permutation(600).astype(np.int32)
    d_old, d_table, d_free, start, d_start = i32(old), i32(table), i32(free), 0, None
    for _ in range(10):
        new = rng.integers(0, 20, n_req)
        n_tokens = int(new.sum()) + 3
        length, cu, slots, positions, counts, table = plan_loops(old, new, table, free, n_tokens, page, start)
        got = smla.sparse_mla_plan_pages(d_old, i32(new), d_table, d_free, n_tokens, page_block=page, free_start=d_start)
        for g, w in zip(got, (length, cu, slots, positions, counts)):
            assert g.tolist() == list(w)
        assert np.array_equal(d_table.cpu().numpy(), table)
        old, start = np.asarray(length), counts[1]
        d_old, d_start = got[0], got[4][1:2].clone()


def test_plan_refuses_overlapping_and_wrong_tensors():
    a, t, f = i32([1, 2]), i32([[0], [1]]), i32([2, 3, 4])
    with pytest.raises(smla.SmlaError):
        smla.sparse_mla_plan_pages(a, i32([1, 1]), t, f, 2, seqlens_k=a)
    counts = i32([0, 0, 0])
    with pytest.raises(smla.SmlaError):
        smla.sparse_mla_plan_pages(a, i32([1, 1]), t, f, 2, free_start=counts[1:2], counts=counts)
    with pytest.raises(ValueError):
        smla.sparse_mla_plan_pages(a, i32([1]), t, f, 2)
    with pytest.raises(ValueError):
        smla.sparse_mla_plan_pages(a, i32([1, 1]), t.t(), f, 2)
    with pytest.raises(ValueError):
        smla.sparse_mla_plan_pages(a, i32([1, 1]), t, f, -1)
    with pytest.raises(ValueError):
        smla.sparse_mla_plan_pages(a, i32([1, 1]), t, f, 2, slots=i32([0, 0, 0]))


# --------------------------------------------------------------------------------- row append
def rope_table(max_pos):
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    return torch.cat([angle.cos(), angle.sin()], 1).float().cuda()


def turned64(x, cs, sn):
    """The rotation, and the sum of its terms' magnitudes."""
    x = x.double()
    a, b = x[..., 0::2], x[..., 1::2]
    val = torch.stack([a * cs - b * sn, b * cs + a * sn], -1).flatten(-2)
    mag = torch.stack([(a * cs).abs() + (b * sn).abs(), (b * cs).abs() + (a * sn).abs()], -1).flatten(-2)
    return val, mag


@pytest.mark.parametrize("n", [1, 7, 300])
@pytest.mark.parametrize("d_qk,norm,roped,heads", [
    (512, True, False, 0), (512, False, False, 0), (576, True, True, 0), (576, False, True, 1), (576, True, True, 20),
    (576, True, False, 0), (576, False, False, 0), (576, True, True, 128),
])
def test_append_against_64_bits(n, d_qk, norm, roped, heads):
    g = torch.Generator().manual_seed(n * 1000 + d_qk + heads)

    def normal(*shape):
        return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()

    rows, max_pos = 400, 50
    x = normal(n, d_qk + 24)
    c, k = x[:, :512], x[:, 512:576] if d_qk == 576 else None
    pool, w = normal(rows, 1, d_qk), normal(512) if norm else None
    slots = torch.randperm(rows, generator=g)[:n].to(torch.int32)
    positions = torch.randint(0, max_pos, (n,), generator=g).to(torch.int32)
    if n > 5:
        slots[1], slots[2], positions[3], positions[4] = -1, rows, -1, max_pos
    q_pe = normal(n, heads, 192)[..., 128:] if heads else None
    q = normal(n, heads, 576) if heads else None
    table = rope_table(max_pos) if roped else None
    want, tol = pool.double(), torch.zeros_like(pool, dtype=torch.float64)
    want_q, tol_q = (q.double(), torch.zeros_like(q, dtype=torch.float64)) if heads else (None, None)
    c64 = c.double()
    y = c64 / (c64.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double() if norm else c64
    # one rounding to bf16; before it the mean (512 terms), its square root and two products in fp32
    y_tol = y.abs() * (U16 + 520 * U32) if norm else y * 0
    for t in range(n):
        pos = int(positions[t])
        if roped and not 0 <= pos < max_pos:
            continue
        cs, sn = (table[pos, :32].double(), table[pos, 32:].double()) if roped else (None, None)
        if heads:
            val, mag = turned64(q_pe[t], cs, sn)
            want_q[t, :, 512:], tol_q[t, :, 512:] = val, val.abs() * U16 + mag * 4 * U32
        if not 0 <= int(slots[t]) < rows:
            continue
        s = int(slots[t])
        want[s, 0, :512], tol[s, 0, :512] = y[t], y_tol[t]
        if d_qk == 576:
            val, mag = turned64(k[t], cs, sn) if roped else (k[t].double(), k[t].double() * 0)
            want[s, 0, 512:], tol[s, 0, 512:] = val, (val.abs() * U16 + mag * 4 * U32 if roped else 0.0)
    got = smla.sparse_mla_append_kv(c, k, slots.cuda(), pool, norm_weight=w, positions=positions.cuda(), rope=table,
                                    q_pe=q_pe, q=q)
    assert got is pool
    assert bool(((pool.double() - want).abs() <= tol).all())    # rows of no token: equal
    if heads:
        assert bool(((q.double() - want_q).abs() <= tol_q).all())


def test_append_turns_the_queries_in_place():
    torch.manual_seed(0)
    n, h = 9, 33
    q = torch.randn(n, h, 576, device="cuda").to(torch.bfloat16)
    q2, before = q.clone(), q.clone()
    x, pool = torch.randn(n, 576, device="cuda").to(torch.bfloat16), torch.zeros(64, 1, 576, device="cuda", dtype=torch.bfloat16)
    pos, slots, table = i32(np.arange(n)), i32(np.arange(n)), rope_table(32)
    smla.sparse_mla_append_kv(x[:, :512], x[:, 512:], slots, pool, positions=pos, rope=table, q_pe=before[..., 512:], q=q2)
    smla.sparse_mla_append_kv(x[:, :512], x[:, 512:], slots, pool, positions=pos, rope=table, q_pe=q[..., 512:], q=q)
    assert torch.equal(q, q2) and torch.equal(q[0], before[0]) and not torch.equal(q, before)


def test_append_writes_rows_past_2_gib():
    rows = 2_000_000
    pool = torch.zeros(rows, 1, 576, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(3, 576, device="cuda").to(torch.bfloat16)
    smla.sparse_mla_append_kv(x[:, :512], x[:, 512:], i32([rows - 1, 5, 1_900_001]), pool)
    assert torch.equal(pool[rows - 1, 0], x[0]) and torch.equal(pool[5, 0], x[1]) and torch.equal(pool[1_900_001, 0], x[2])
    assert int((pool != 0).any(-1).sum()) == 3


def test_append_refuses_wrong_tensors():
    x = torch.zeros(4, 576, device="cuda", dtype=torch.bfloat16)
    pool, s = torch.zeros(8, 1, 576, device="cuda", dtype=torch.bfloat16), i32([0, 1, 2, 3])
    c, k, table, q = x[:, :512], x[:, 512:], rope_table(4), torch.zeros(4, 2, 576, device="cuda", dtype=torch.bfloat16)
    for kw in (dict(k_pe=None), dict(k_pe=k[:3]), dict(c_kv=c[:, ::2]), dict(rope=table), dict(rope=table[:, :32], positions=s),
               dict(rope=table, positions=s, q=q), dict(q_pe=q[..., 512:], q=q), dict(norm_weight=c[0, :100]),
               dict(rope=table, positions=s, q_pe=q[..., 512:], q=q[:, :1]), dict(slots=s[:3]),
               dict(c_kv=x.view(-1)[4:4 + 3 * 576].view(3, 576)[:, :512], k_pe=k[:3], slots=s[:3])):
        a = dict(c_kv=c, k_pe=k, slots=s, kv_pool=pool)
        a.update(kw)
        with pytest.raises((ValueError, smla.SmlaError)):
            smla.sparse_mla_append_kv(**a)
    with pytest.raises(smla.SmlaError):   # rows on top of the input
        smla.sparse_mla_append_kv(pool[4:, 0, :512], k, s, pool)
    assert int(pool.count_nonzero()) == 0


# ---------------------------------------------------------------------- dense chunk attention
def chunk_case(seed, q_lens, k_lens, heads, d_qk=576, page=64, scale=1.0, spare=2, tail=0, width=None):
    """Random requests; every pool row that no request's key occupies is NaN."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-k // page) for k in k_lens]
    n_pages = sum(held) + 3
    width = max(held + [0]) + spare if width is None else width
    pages = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((len(q_lens), width), -1, dtype=torch.int32)
    pool = torch.full((n_pages * page, 1, d_qk), float("nan"), dtype=torch.bfloat16)
    at = 0
    for b, k in enumerate(k_lens):
        mine = pages[at:at + held[b]]
        at += held[b]
        table[b, :min(held[b], width)] = mine[:width]
        rows = (mine.long()[:, None] * page + torch.arange(page)).reshape(-1)[:k]
        pool[rows, 0] = (torch.randn(k, d_qk, generator=g) * scale).to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    q = (torch.randn(int(cu[-1]) + tail, heads, d_qk, generator=g) * scale).to(torch.bfloat16)
    return dict(q=q.cuda(), kv_pool=pool.cuda(), block_table=table.cuda(), cu_seqlens_q=i32(cu), seqlens_k=i32(k_lens),
                page_block=page)


def chunk_check(w, causal=True, sink=None, sm_scale=None, run=None, **kw):
    """The operator against 64 bits, request by request, within the bound of its roundings."""
    q, cu, page = w["q"], w["cu_seqlens_q"].tolist(), w["page_block"]
    n, h, d = q.shape
    scale = d ** -0.5 if sm_scale is None else sm_scale
    mark = dict(out=torch.full((n, h, 512), 3.0, dtype=torch.bfloat16, device="cuda"),
                lse=torch.full((n, h), 5.0, device="cuda"), max_logits=torch.full((n, h), 7.0, device="cuda"))
    got = (run or smla.sparse_mla_chunk_fwd_paged)(**w, causal=causal, attn_sink=sink, sm_scale=sm_scale, **mark, **kw)
    out, lse, top = got
    covered = torch.zeros(n, dtype=torch.bool, device="cuda")
    table, rows_total = w["block_table"].long(), w["kv_pool"].shape[0]
    for b, n_k in enumerate(w["seqlens_k"].tolist()):
        t0, t1, n_k = cu[b], cu[b + 1], max(n_k, 0)
        covered[t0:t1] = True
        if t1 == t0:
            continue
        j = torch.arange(n_k, device="cuda")
        col = j // page
        entry = torch.where(col < table.shape[1], table[b, col.clamp(max=table.shape[1] - 1)], -1)
        row = entry * page + j % page
        ok = (entry >= 0) & (row < rows_total)
        kv = torch.where(ok[:, None], w["kv_pool"][row.clamp(0, rows_total - 1), 0].double(), 0.0)
        for a in range(t0, t1, 64):
            e = min(a + 64, t1)
            qt = q[a:e].double()
            s = torch.einsum("thd,kd->thk", qt, kv) * scale
            # fp32 sums of d products: d 2^-23 of the sum of magnitudes, whatever the order and the
            # rounding of the additions
            ds = float((torch.einsum("thd,kd->thk", qt.abs(), kv.abs()) * scale).max() if n_k else 0.0) * d * 2 * U32
            seen = ok[None, :].expand(e - a, -1)
            if causal:
                seen = seen & (j[None, :] <= (torch.arange(a, e, device="cuda") - t1 + n_k)[:, None])
            s = s.masked_fill(~seen[:, None, :], float("-inf"))
            empty = ~seen.any(-1)
            live = ~empty
            assert bool((out[a:e][empty] == 0).all()) and not bool(torch.signbit(out[a:e][empty]).any())
            assert bool((lse[a:e][empty] == float("inf")).all()) and bool((top[a:e][empty] == float("-inf")).all())
            if not bool(live.any()):
                continue
            s = s[live]
            m, z = s.max(-1).values, torch.logsumexp(s, -1)
            full = z if sink is None else torch.logaddexp(z, sink.double()[None])
            p = (s - full[..., None]).exp()
            o = torch.einsum("thk,kd->thd", p, kv[:, :512])
            mag = torch.einsum("thk,kd->thd", p, kv[:, :512].abs())
            # weights: one rounding to bf16, the logits' error in numerator and denominator, the
            # exponential and the sums of n_k terms in fp32; then the output's own rounding
            tol = mag * (U16 + 2.1 * ds + 2 * (n_k + 16) * U32) * (1 + U16) + o.abs() * U16 + 1e-30
            bad = ((out[a:e][live].double() - o).abs() - tol).max()
            assert float(bad) <= 0, f"request {b}: out off by {float(bad):.3e} more than {float(tol.max()):.3e}"
            e_m = float((top[a:e][live].double() - m).abs().max())
            assert e_m <= ds + 4 * U32 * float(m.abs().max()), f"request {b}: max_logits off by {e_m:.3e}"
            e_l = float((lse[a:e][live].double() - z).abs().max())
            assert e_l <= ds + (n_k + 16) * U32 + 8 * U32 * float(z.abs().max()) + 8 * U32, f"request {b}: lse off by {e_l:.3e}"
    # rows of no request are left as they were
    assert bool((out[~covered] == 3.0).all()) and bool((lse[~covered] == 5.0).all()) and bool((top[~covered] == 7.0).all())
    return got


@pytest.mark.parametrize("heads", [1, 16, 20, 64, 96, 128, 129, 192, 320])
@pytest.mark.parametrize("d_qk", [512, 576])
def test_chunk_heads(heads, d_qk):
    chunk_check(chunk_case(heads, [1, 3, 10], [77, 3, 200], heads, d_qk))


@pytest.mark.parametrize("page", [1, 4, 7, 8, 16, 24, 32, 48, 64, 100, 128, 256])
def test_chunk_pages(page):
    chunk_check(chunk_case(page, [2, 9, 1], [130, 65, 300], 16, page=page))
    chunk_check(chunk_case(page + 1, [5, 1], [64, 129], 128, 512, page=page), causal=False)


@pytest.mark.parametrize("n_k", [1, 2, 15, 31, 32, 33, 47, 48, 63, 64, 65, 95, 96, 97, 127, 128, 129, 191, 193, 255, 257, 1000])
def test_chunk_key_counts(n_k):
    chunk_check(chunk_case(n_k, [1], [n_k], 128))
    chunk_check(chunk_case(n_k, [min(n_k, 40)], [n_k], 32))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("sink", [True, False])
@pytest.mark.parametrize("heads,d_qk", [(16, 576), (20, 512), (128, 576), (200, 576)])
def test_chunk_ragged(causal, sink, heads, d_qk):
    w = chunk_case(heads, [0, 17, 1, 0, 64, 5, 130], [40, 17, 900, 0, 333, 5, 200], heads, d_qk, tail=3)
    s = torch.randn(heads, device="cuda") * 3 if sink else None
    chunk_check(w, causal, s)


def test_chunk_rows_that_see_nothing():
    # more new tokens than keys, no keys at all, a negative length; behind them an ordinary request
    w = chunk_case(3, [9, 4, 2, 6], [5, 0, 0, 50], 48)
    w["seqlens_k"][2] = -3
    for sink in (None, torch.randn(48, device="cuda")):
        chunk_check(w, True, sink)
        chunk_check(w, False, sink)


def test_chunk_sink_of_any_size():
    w = chunk_case(4, [3, 1], [70, 9], 6)
    chunk_check(w, True, torch.tensor([float("-inf"), -100.0, -1.0, 0.0, 30.0, 80.0], device="cuda"))


@pytest.mark.parametrize("heads", [16, 128])
def test_chunk_unmapped_pages(heads):
    w = chunk_case(6, [4, 3, 30], [400, 500, 130], heads, page=16)
    w["block_table"][0, 3] = -1
    w["block_table"][0, 20:] = -7
    w["block_table"][1, :] = 2 ** 30           # past the pool
    w["block_table"][2, 1] = w["kv_pool"].shape[0] // 16
    w["block_table"][2, 8] = -1                # the new tokens' own last page
    chunk_check(w)
    chunk_check(w, causal=False)


def test_chunk_table_shorter_than_the_keys():
    w = chunk_case(7, [4, 20], [300, 20], 32, page=16, width=10)
    chunk_check(w)
    chunk_check(w, causal=False)


def test_chunk_large_scores():
    # scores of a thousand and more: the running maximum moves far, block after block
    w = chunk_case(8, [3, 40], [700, 650], 16, scale=12.0)
    chunk_check(w)
    w = chunk_case(9, [2], [2000], 128, scale=0.01)
    chunk_check(w, sm_scale=3.0)


def test_chunk_ascending_scores():
    """Every later key scores higher than all before it: the running maximum moves in every block."""
    w = chunk_case(10, [2], [1500], 128)
    w["q"][:] = 1.0
    rows = torch.arange(1500, device="cuda")
    pool_rows = (w["block_table"][0].long()[rows // 64] * 64 + rows % 64)
    w["kv_pool"][pool_rows, 0] = ((rows[:, None] - 700) * 0.002).to(torch.bfloat16).expand(-1, 576)
    chunk_check(w)


@pytest.mark.parametrize("shape", [([1] * 300, [50 + 7 * i for i in range(300)], 16), ([1], [20000], 128),
                                   ([1], [20000], 16), ([3, 1, 2], [9000, 11, 5000], 128), ([600], [2500], 64),
                                   ([1000, 1], [1000, 3], 20), ([2] * 40, [1024] * 40, 128)])
def test_chunk_splits_and_joins(shape):
    """Sizes where requests are cut over workers and joined, evenly and not."""
    q_lens, k_lens, heads = shape
    chunk_check(chunk_case(len(q_lens), q_lens, k_lens, heads))


def test_chunk_many_requests():
    rng = np.random.default_rng(2)
    q_lens = rng.integers(0, 3, 3000)
    chunk_check(chunk_case(12, q_lens.tolist(), (q_lens + rng.integers(0, 40, 3000)).tolist(), 4, 512, page=8))


def test_chunk_pool_past_2_gib():
    rows = 2_500_032
    pool = torch.empty(rows, 1, 576, device="cuda", dtype=torch.bfloat16).normal_()
    table = i32(np.array([[rows // 64 - 1, 3, rows // 64 - 2, 39000, 20]]))
    w = dict(q=torch.randn(2, 128, 576, device="cuda").to(torch.bfloat16), kv_pool=pool, block_table=table,
             cu_seqlens_q=i32([0, 2]), seqlens_k=i32([300]), page_block=64)
    chunk_check(w)


def test_chunk_sums_past_their_bounds_stay_inside():
    """cu_seqlens_q that runs past the tensors is clamped: no row outside q is touched."""
    w = chunk_case(13, [4, 4], [90, 70], 16)
    big = torch.full((24, 16, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    w["cu_seqlens_q"] = i32([-5, 4, 1000])
    out, lse, top = smla.sparse_mla_chunk_fwd_paged(**w, out=big[8:16])
    torch.cuda.synchronize()
    assert bool((big[:8] == 3).all()) and bool((big[16:] == 3).all()) and bool(torch.isfinite(lse[:4]).all())


def test_chunk_twice_the_same_bits_and_two_streams():
    w = chunk_case(14, [1, 300, 2], [5000, 400, 3001], 128)
    a = smla.sparse_mla_chunk_fwd_paged(**w)
    b = smla.sparse_mla_chunk_fwd_paged(**w)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    many = [smla.sparse_mla_chunk_fwd_paged(**w, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    for other in [b, *many]:
        assert all(torch.equal(x, y) for x, y in zip(a, other))


def test_chunk_workspace_of_the_caller():
    w = chunk_case(15, [1, 1], [5000, 700], 128)
    need = smla.load_library().sparse_mla_chunk_workspace_size(2, 128)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda")
    got = chunk_check(w, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(got, smla.sparse_mla_chunk_fwd_paged(**w)))
    if need:
        with pytest.raises(smla.SmlaError):
            smla.sparse_mla_chunk_fwd_paged(**w, workspace=ws[:need - 256])
        with pytest.raises(smla.SmlaError):
            smla.sparse_mla_chunk_fwd_paged(**w, workspace=ws[16:])


def test_chunk_in_graphs_with_changing_lengths():
    """Two captured calls with a workspace each, replayed after the lengths changed in place."""
    ws = [chunk_case(16 + i, [1, 20], [900, 600], 128) for i in range(2)]
    graphs, outs = [], []
    for w in ws:
        smla.sparse_mla_chunk_fwd_paged(**w)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(smla.sparse_mla_chunk_fwd_paged(**w))
        graphs.append(g)
    for lens, cu in (([900, 600], [0, 1, 21]), ([40, 333], [0, 1, 21]), ([900, 20], [0, 3, 21]), ([0, 600], [0, 0, 21])):
        for w in ws:
            w["seqlens_k"].copy_(i32(lens))
            w["cu_seqlens_q"].copy_(i32(cu))
        for g in graphs:
            g.replay()
        for w, o in zip(ws, outs):
            chunk_check(w, run=lambda o=o, **kw: [dst.copy_(src) for dst, src in zip((kw["out"], kw["lse"], kw["max_logits"]), o)])


def test_chunk_refuses_wrong_tensors():
    w = chunk_case(18, [2], [70], 16)
    for kw in (dict(seqlens_k=i32([1, 2])), dict(cu_seqlens_q=i32([0, 1, 2])), dict(block_table=w["block_table"][0]),
               dict(kv_pool=w["kv_pool"][..., :512].contiguous()), dict(attn_sink=torch.zeros(3, device="cuda")),
               dict(q=w["q"][:, 0]), dict(q=w["q"].transpose(0, 1)), dict(d_v=256), dict(sm_scale=-1.0), dict(page_block=0),
               dict(out=torch.zeros(2, 16, 576, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises((ValueError, smla.SmlaError)):
            smla.sparse_mla_chunk_fwd_paged(**dict(w, **kw))


# ------------------------------------------------------------------------------ a serving step
def test_serving_steps_together():
    """Three steps (prompts, a mixed step, decode): plan, append, attend.  The cache that the steps
    build is compared with one built in 64 bits; the dense attention with 64 bits on that cache,
    and with the sparse form given every position."""
    torch.manual_seed(3)
    n_req, heads, page, width, layers = 5, 64, 16, 24, 2
    table, free = torch.full((n_req, width), -1, dtype=torch.int32, device="cuda"), i32(np.random.default_rng(1).permutation(90))
    pools = [torch.full((90 * page, 1, 576), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
    rope, seqlens, start = rope_table(1024), i32([0] * n_req), None
    w = (1 + 0.1 * torch.randn(512, device="cuda")).to(torch.bfloat16)
    for new in ([100, 33, 1, 64, 7], [1, 40, 1, 0, 100], [1, 1, 1, 1, 1]):
        n = sum(new) + 2
        seqlens_k, cu, slots, positions, counts = smla.sparse_mla_plan_pages(
            seqlens, i32(new), table, free, n, page_block=page, free_start=start)
        for pool in pools:
            x = torch.randn(n, 576, device="cuda").to(torch.bfloat16)
            q, q_pe = torch.randn(n, heads, 576, device="cuda").to(torch.bfloat16), torch.randn(n, heads, 64, device="cuda").to(torch.bfloat16)
            smla.sparse_mla_append_kv(x[:, :512], x[:, 512:], slots, pool, norm_weight=w, positions=positions, rope=rope,
                                      q_pe=q_pe, q=q)
            args = dict(q=q, kv_pool=pool, block_table=table, cu_seqlens_q=cu, seqlens_k=seqlens_k, page_block=page)
            out, lse, top = chunk_check(args)
            # the sparse form with every visible position in its list, request by request
            for b in range(n_req):
                t0, t1, n_k = int(cu[b]), int(cu[b + 1]), int(seqlens_k[b])
                if t1 == t0:
                    continue
                last = torch.arange(n_k - (t1 - t0), n_k, device="cuda")
                j = torch.arange(n_k, device="cuda")
                idx = torch.where(j[None] <= last[:, None], j[None], -1).to(torch.int32)[:, None].contiguous()
                o2, l2, m2 = smla.sparse_mla_fwd_paged(q[t0:t1], pool, table[b:b + 1], idx, page_block=page,
                                                       s_q_per_req=t1 - t0)
                assert float((lse[t0:t1] - l2).abs().max()) < 1e-3 and float((top[t0:t1] - m2).abs().max()) < 1e-3
                # each side is within 2.1 roundings to bf16 of a weighted mean of |v| <= max |v|
                assert float((out[t0:t1].float() - o2.float()).abs().max()) <= 4.2 * U16 * float(pool[table[b][table[b] >= 0].long()[:, None] * page].float().nan_to_num().abs().max().clamp(min=5.0))
        assert int(counts[0]) == sum(new) and int(counts[2]) == 0
        seqlens, start = seqlens_k, counts[1:2].clone()


def test_chunk_batch_with_empty_slots():
    """Many request slots, few of them with tokens: at the front, scattered, and at the end."""
    for seed, live in ((0, range(5)), (1, range(3, 900, 97)), (2, [899]), (3, [])):
        q_lens, k_lens = [0] * 900, [11] * 900
        for i in live:
            q_lens[i], k_lens[i] = 1 + i % 3, 50 + i
        chunk_check(chunk_case(seed, q_lens, k_lens, 16, 512, page=16, tail=2))


def test_chunk_of_1024_heads():
    chunk_check(chunk_case(20, [2, 1], [140, 33], 1024, 512))


FIRST_CALLS_CAPTURED = """
import sys
sys.path.insert(0, sys.argv[1])
import torch, sparse_mla_attention_fwd_gb300 as smla
torch.manual_seed(0)
pool = torch.randn(4 * 64, 1, 576, device="cuda").to(torch.bfloat16)
q, x = (torch.randn(*s, device="cuda").to(torch.bfloat16) for s in ((3, 16, 576), (3, 576)))
lens, new, free = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([100, 64], [2, 1], [3, 2]))
table = torch.tensor([[0, 1, -1], [2, -1, -1]], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
def step():
    k, cu, slots, pos, counts = smla.sparse_mla_plan_pages(lens, new, table, free, 3)
    smla.sparse_mla_append_kv(x[:, :512], x[:, 512:], slots, pool)
    return smla.sparse_mla_chunk_fwd_paged(q, pool, table, cu, k)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = step()
graph.replay()
torch.cuda.synchronize()
captured = [t.clone() for t in captured]
assert all(torch.equal(a, b) for a, b in zip(captured, step())) and smla.sparse_mla_device_status() == 0
"""


def test_first_calls_of_a_process_may_be_captured():
    done = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED, ROOT], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_a_whole_step_in_one_graph():
    """Plan, append and attend captured once; replayed over steps whose lengths, free list position and
    inputs change in place, against the same steps run call by call."""
    torch.manual_seed(4)
    n_req, heads, page, width, n, steps = 6, 16, 16, 12, 64, ([20, 0, 7, 1, 16, 3], [1, 33, 1, 0, 1, 20], [1] * 6, [0] * 6)
    free, rope = i32(np.random.default_rng(2).permutation(60)), rope_table(256)

    def fresh():
        return dict(lens=i32([0] * n_req), new=i32([0] * n_req), start=i32([0]), table=i32(np.full((n_req, width), -1)),
                    pool=torch.zeros(60 * page, 1, 576, dtype=torch.bfloat16, device="cuda"),
                    x=torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda"),
                    q=torch.zeros(n, heads, 576, dtype=torch.bfloat16, device="cuda"))

    def step(s):
        k, cu, slots, pos, counts = smla.sparse_mla_plan_pages(s["lens"], s["new"], s["table"], free, n, page_block=page,
                                                               free_start=s["start"])
        smla.sparse_mla_append_kv(s["x"][:, :512], s["x"][:, 512:], slots, s["pool"], positions=pos, rope=rope,
                                  q_pe=s["q"][..., 512:], q=s["q"])
        got = smla.sparse_mla_chunk_fwd_paged(s["q"], s["pool"], s["table"], cu, k, page_block=page)
        s["lens"].copy_(k)
        s["start"].copy_(counts[1:2])
        return (*got, slots, pos, counts)

    a, b = fresh(), fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(b)
    for new in steps:
        x, q = torch.randn(n, 576, device="cuda"), torch.randn(n, heads, 576, device="cuda")
        for s in (a, b):
            s["new"].copy_(i32(new))
            s["x"].copy_(x)
            s["q"].copy_(q)
        want = step(a)
        graph.replay()
        used = sum(new)
        assert all(torch.equal(u[:used], v[:used]) for u, v in zip(want[:3], captured[:3]))
        assert all(torch.equal(u, v) for u, v in zip(want[3:], captured[3:]))
        assert all(torch.equal(a[key], b[key]) for key in ("lens", "start", "table", "pool", "q"))
    assert int(captured[5][2]) == 0


def test_threads_call_at_once():
    """Four threads, a stream each, over one cache."""
    w = chunk_case(21, [1, 40, 3], [3000, 400, 901], 64)
    want = smla.sparse_mla_chunk_fwd_paged(**w)
    torch.cuda.synchronize()
    same = []

    def work():
        s = torch.cuda.Stream()
        got = [smla.sparse_mla_chunk_fwd_paged(**w, stream=s) for _ in range(20)]
        s.synchronize()
        same.append(all(torch.equal(x, y) for g in got for x, y in zip(want, g)))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert same == [True] * 4


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("q_lens,k_lens,heads,d_qk", [([3], [70], 4, 576), ([1], [9000], 4, 576), ([40, 1], [700, 5000], 128, 512),
                                                      ([2, 3], [900, 70], 200, 576)])
def test_chunk_nan_queries_stay_visible(bad, q_lens, k_lens, heads, d_qk):
    """A broken query gives NaN, not the values of a row that sees no key; every other row keeps its bits.  Whole tiles and
    cut ones.  (An infinite column gives scores of both infinities, whose sum is NaN.)"""
    w = chunk_case(heads, q_lens, k_lens, heads, d_qk)
    sink = torch.randn(heads, device="cuda")
    want = smla.sparse_mla_chunk_fwd_paged(**w, attn_sink=sink)
    broken = torch.zeros(w["q"].shape[:2], dtype=torch.bool, device="cuda")
    broken[0, 1] = broken[-1, heads - 1] = True
    w["q"][..., 5] = torch.where(broken, bad, w["q"][..., 5])
    got = smla.sparse_mla_chunk_fwd_paged(**w, attn_sink=sink)
    for g, x in zip(got, want):
        assert bool(g[broken].isnan().all())
        assert torch.equal(g[~broken], x[~broken])


def test_chunk_nan_keys_reach_the_tokens_that_see_them():
    for n_k in (100, 9000):
        w = chunk_case(22, [4, 2], [n_k, 90], 16)
        at = n_k - 3                                   # the second token's own position
        w["kv_pool"][w["block_table"][0, at // 64].long() * 64 + at % 64, 0, 7] = float("nan")
        out, lse, top = smla.sparse_mla_chunk_fwd_paged(**w)
        assert all(bool(x[1:4].isnan().all()) for x in (lse, top)) and bool(out[1:4].isnan().any(-1).all())
        assert all(bool(torch.isfinite(x[4:].float()).all()) for x in (out, lse, top))


def test_chunk_nan_does_not_hide_empty_rows():
    w = chunk_case(23, [5, 3], [2, 0], 16)             # the first three tokens, and all of the second request, see no key
    w["q"][:] = float("nan")
    out, lse, top = smla.sparse_mla_chunk_fwd_paged(**w)
    for rows in (slice(0, 3), slice(5, 8)):
        assert bool((out[rows] == 0).all()) and bool((lse[rows] == float("inf")).all()) and bool((top[rows] == float("-inf")).all())
    assert all(bool(x[3:5].isnan().all()) for x in (out, lse, top))


def test_a_request_that_outgrows_the_rope_table():
    """Plan, append and attend across the end of the rope table: the tokens behind it are counted, call after call and
    in a replayed graph; with a table for every position of the block table no row that is read stays unwritten."""
    torch.manual_seed(6)
    heads, page, width, n = 16, 16, 4, 90
    lens, new = i32([30, 0, 61]), i32([20, 64, 5])     # positions to 49, 63 and 65: the last two past the block table
    x, q = torch.randn(n, 576, device="cuda").to(torch.bfloat16), torch.randn(n, heads, 576, device="cuda").to(torch.bfloat16)
    for max_pos, past in ((64, 2), (40, 10 + 24 + 5), (66, 0), (63, 1 + 3)):
        table = i32([[0, 1, -1, -1], [-1] * 4, [2, 3, 4, 5]])
        pool = torch.full((20 * page, 1, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
        k, cu, slots, pos, counts = smla.sparse_mla_plan_pages(lens, new, table, i32(np.arange(6, 20)), n, page_block=page)
        old = torch.cat([table[0, :2].long()[:, None] * page + torch.arange(page, device="cuda"),
                         table[2].long()[:, None] * page + torch.arange(page, device="cuda")]).flatten()
        pool[old] = 1.0
        pool[slots[slots >= 0].long()] = float("nan")
        beyond, turned = torch.zeros(1, dtype=torch.int32, device="cuda"), q.clone()
        args = dict(c_kv=x[:, :512], k_pe=x[:, 512:], slots=slots, kv_pool=pool, positions=pos, rope=rope_table(max_pos),
                    q_pe=q[..., 512:], q=turned)
        smla.sparse_mla_append_kv(**args, past_rope=beyond)
        assert int(beyond) == past
        smla.sparse_mla_append_kv(**args, past_rope=beyond, stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            smla.sparse_mla_append_kv(**args, past_rope=beyond)
        graph.replay()
        assert int(beyond) == 3 * past
        written = int((~pool[slots[slots >= 0].long(), 0].isnan().any(-1)).sum())
        assert written == int(((pos >= 0) & (pos < max_pos) & (slots >= 0)).sum())
        if max_pos >= width * page:
            chunk_check(dict(q=turned, kv_pool=pool, block_table=table, cu_seqlens_q=cu, seqlens_k=k, page_block=page))
    with pytest.raises(ValueError):
        smla.sparse_mla_append_kv(**args, past_rope=i32([0, 0]))
    with pytest.raises(smla.SmlaError):
        smla.sparse_mla_append_kv(**args, past_rope=pool.view(torch.int32).view(-1)[:1])


def test_append_of_one_token_or_head_with_any_stride():
    """A projection of one column vector, transposed, is contiguous and has the strides (1, 1)."""
    torch.manual_seed(7)
    up, hidden = torch.randn(576 + 192, 64, device="cuda").to(torch.bfloat16), torch.randn(64, 1, device="cuda").to(torch.bfloat16)
    y = (up @ hidden).t()
    assert y.stride() == (1, 1)
    slots, pos, rope = i32([3]), i32([5]), rope_table(9)
    got = []
    for c_stride, k_stride, q_stride in ((1, 3, 7), (512, 64, 192)):
        pool, q = torch.zeros(8, 1, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 3, 576, dtype=torch.bfloat16, device="cuda")
        smla.sparse_mla_append_kv(y[:, :512].as_strided((1, 512), (c_stride, 1)), y[:, 512:576].as_strided((1, 64), (k_stride, 1)),
                                  slots, pool, positions=pos, rope=rope, q_pe=y[:, 576:].as_strided((1, 3, 64), (q_stride, 64, 1)), q=q)
        got.append((pool, q))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and int((got[0][0] != 0).any(-1).sum()) == 1
    x, one = torch.randn(4, 576, device="cuda").to(torch.bfloat16), torch.randn(4, 1, 64, device="cuda").to(torch.bfloat16)
    got = []
    for qp in (one, one.as_strided((4, 1, 64), (64, 3, 1))):
        pool, q = torch.zeros(8, 1, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 1, 576, dtype=torch.bfloat16, device="cuda")
        smla.sparse_mla_append_kv(x[:, :512], x[:, 512:], i32([0, 1, 2, 7]), pool, positions=i32([0, 1, 8, 3]), rope=rope, q_pe=qp, q=q)
        got.append((pool, q))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_chunk_buffers_may_touch_and_not_overlap():
    w = chunk_case(24, [2, 1], [700, 90], 16, 512)
    want = smla.sparse_mla_chunk_fwd_paged(**w)
    rows, need = 3 * 16, smla.load_library().sparse_mla_chunk_workspace_size(3, 16)
    block = torch.empty(need + rows * (1024 + 1024 + 8), dtype=torch.uint8, device="cuda")
    ws, q, out, lse, top = block.split([need, rows * 1024, rows * 1024, rows * 4, rows * 4])
    q, out = q.view(torch.bfloat16).view(3, 16, 512), out.view(torch.bfloat16).view(3, 16, 512)
    lse, top = lse.view(torch.float32).view(3, 16), top.view(torch.float32).view(3, 16)
    q.copy_(w["q"])
    w["q"] = q
    got = smla.sparse_mla_chunk_fwd_paged(**w, out=out, lse=lse, max_logits=top, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(got[0], out)
    for kw in (dict(out=q), dict(lse=top), dict(workspace=block[256:256 + need]), dict(out=w["kv_pool"][:rows].view(3, 16, 512))):
        with pytest.raises(smla.SmlaError):
            smla.sparse_mla_chunk_fwd_paged(**w, **dict(dict(out=out, lse=lse, max_logits=top, workspace=ws), **kw))


def test_chunk_waits_give_up_and_report_it():
    """A wait that runs out is reported by the chunk kernel's word and by the Python function, until it is reset; the
    other kernels' word stays clear, and the next call is right."""
    lib, limit = smla.load_library(), 20_000_000
    assert smla.sparse_mla_device_status(reset=True) == 0
    e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    stream = torch.cuda.current_stream()
    e[0].record(stream)
    assert lib.sparse_mla_chunk_selftest_wait_timeout(limit, stream.cuda_stream) == 0
    e[1].record(stream)
    torch.cuda.synchronize()
    # two waits of the limit, 16 tries of 0.1 ms after it at most; the third at once instead of after its 2 s
    assert 40.0 <= e[0].elapsed_time(e[1]) < 1000.0
    assert lib.sparse_mla_device_status(0) == 0 and lib.sparse_mla_chunk_device_status(0) == 5
    assert smla.sparse_mla_device_status() == 5
    assert smla.sparse_mla_device_status(reset=True) == 5
    assert smla.sparse_mla_device_status() == 0 and lib.sparse_mla_chunk_device_status(0) == 0
    assert lib.sparse_mla_selftest_wait_timeout(limit, None) == 0      # the other word, by the same function
    torch.cuda.synchronize()
    assert lib.sparse_mla_chunk_device_status(0) == 0 and smla.sparse_mla_device_status(reset=True) == 5
    chunk_check(chunk_case(25, [2, 1], [700, 90], 16))


@pytest.mark.parametrize("heads,n_k", [(16, 700), (128, 2600), (20, 9000)])
def test_chunk_large_scores_that_are_exact(heads, n_k):
    """Scores of a thousand and more from small whole numbers, whose products and sums fp32 holds exactly: what is left are
    the roundings of the softmax.  Later keys are longer, so the running maximum moves far, block after block."""
    w = chunk_case(heads, [3], [n_k], heads, page=16)
    g = torch.Generator().manual_seed(n_k)
    length = 1 + torch.arange(n_k) * 6 // n_k
    keys = (torch.randint(-1, 2, (n_k, 576), generator=g) * length[:, None]).to(torch.bfloat16).cuda()
    j = torch.arange(n_k, device="cuda")
    w["kv_pool"][w["block_table"][0, j // 16].long() * 16 + j % 16, 0] = keys
    w["q"] = torch.randint(-12, 13, w["q"].shape, generator=g).to(torch.bfloat16).cuda()
    scale = 0.5
    out, lse, top = smla.sparse_mla_chunk_fwd_paged(**w, sm_scale=scale)
    s = torch.einsum("thd,kd->thk", w["q"].double(), keys.double()) * scale
    s = s.masked_fill(j[None, None] > torch.arange(n_k - 3, n_k, device="cuda")[:, None, None], float("-inf"))
    m, z = s.max(-1).values, torch.logsumexp(s, -1)
    assert float(m.abs().max()) > 1000 and float(s[s > float("-inf")].abs().max()) < 2 ** 22
    assert torch.equal(top.double(), m)
    p = (s - z[..., None]).exp()
    o, mag = torch.einsum("thk,kd->thd", p, keys[:, :512].double()), torch.einsum("thk,kd->thd", p, keys[:, :512].double().abs())
    # The exponents are products with log2 e, and differences of such: four roundings of numbers up to 1.5 max |s|, in base 2,
    # and each move of the running maximum, of which a row has at most one per block, rounds its own once more
    ds = (4 + 2) * 1.5 * float(m.abs().max()) * U32 + n_k / 64 * 4 * U32
    tol = mag * (U16 + 2.1 * ds + 2 * (n_k + 16) * U32) * (1 + U16) + o.abs() * U16 + 1e-30
    assert bool(((out.double() - o).abs() <= tol).all())
    assert float((lse.double() - z).abs().max()) <= ds + (n_k + 16) * U32 + 8 * U32 * float(z.abs().max()) + 8 * U32


WITHOUT_SHORTCUTS = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
if sys.argv[2] == "without":
    sys.modules["torch._C._dynamo.guards"] = None
    del torch._C._cuda_getCurrentRawStream
import sparse_mla_attention_fwd_gb300 as smla
assert (smla._empty_strided.__module__ == smla.__name__) == (sys.argv[2] == "without")
assert (getattr(smla._raw_stream, "__module__", None) == smla.__name__) == (sys.argv[2] == "without")
g = torch.Generator().manual_seed(0)
def normal(*s):
    return torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
pool, q, x = normal(256, 1, 576), normal(3, 16, 576), normal(3, 576)
lens, new, free = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([100, 64], [2, 1], [3, 2]))
table = torch.tensor([[0, 1, -1], [2, -1, -1]], dtype=torch.int32, device="cuda")
side = torch.cuda.Stream()
side.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(side):
    k, cu, slots, pos, counts = smla.sparse_mla_plan_pages(lens, new, table, free, 3)
    smla.sparse_mla_append_kv(x[:, :512], x[:, 512:], slots, pool)
    assert torch.equal(pool[slots.long(), 0], x)
    got = smla.sparse_mla_chunk_fwd_paged(q, pool, table, cu, k)
torch.cuda.synchronize()
torch.save([t.cpu() for t in (k, cu, slots, pos, counts, pool, *got)], sys.argv[3])
"""


def test_wrappers_without_torchs_private_functions(tmp_path):
    """The output allocation and the stream handle through torch's public functions: the same values."""
    got = []
    for mode in ("with", "without"):
        path = str(tmp_path / mode)
        done = subprocess.run([sys.executable, "-c", WITHOUT_SHORTCUTS, ROOT, mode, path], capture_output=True, text=True, timeout=300)
        assert done.returncode == 0, done.stderr[-2000:]
        got.append(torch.load(path))
    assert len(got[0]) == 9 and all(torch.equal(a, b) for a, b in zip(*got))


def test_chunk_scores_past_fp32_are_not_empty_rows():
    """Finite products that the scale takes past fp32's range, whole tiles and cut ones, beside rows that see no key."""
    for k_lens in ([70, 0], [9000, 1]):
        w = chunk_case(26, [2, 3], k_lens, 16)
        w["q"][:2] = w["q"][:2].abs()
        j = torch.arange(k_lens[0], device="cuda")
        rows = w["block_table"][0, j // 64].long() * 64 + j % 64
        w["kv_pool"][rows] = w["kv_pool"][rows].abs() + 0.125        # every score of the first request is above 0
        for sink in (None, torch.randn(16, device="cuda")):
            out, lse, top = smla.sparse_mla_chunk_fwd_paged(**w, sm_scale=2.0 ** 125, attn_sink=sink)
            assert bool(lse[:2].isnan().all()) and bool(out[:2].isnan().all())
            assert not bool(torch.isfinite(top[:2]).any()) and not bool((top[:2] == float("-inf")).any())
            assert bool((out[2:4] == 0).all()) and bool((lse[2:4] == float("inf")).all())
