"""GPU tests of a speculative step's operators: tree planning, tree attention, verification, commit, and steps of all of them
with the paged-cache operators.

References are plain loops (whole numbers and copied rows: equal) or 64-bit torch on the same inputs.  Tolerances count
roundings: u = 2^-8 for one rounding to bf16, 2^-24 for fp32."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import sparse_mla_attention_fwd_gb300 as smla
from test_paged_ops_gpu import chunk_case, i32, rope_table

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U16, U32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(autouse=True)
def device_status():
    yield
    torch.cuda.synchronize()
    assert smla.sparse_mla_device_status() == 0


def random_parents(rng, n, kind="tree"):
    """Parents of n nodes: a chain, a star, a comb (two chains in turn), a tree, or anything (broken entries among them)."""
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1][:n] + [0] * (n - 1)
    if kind == "comb":
        return [i - 2 if i > 1 else i - 1 for i in range(n)]
    tree = [int(rng.integers(max(0, i - 6), i)) if i else -1 for i in range(n)]
    if kind == "any":
        for i in range(n):
            if rng.random() < 0.2:
                tree[i] = int(rng.choice([-1, -7, i, i + 1, n, 2 ** 31 - 1, -2 ** 31]))
    return tree


def ancestors(parents):
    """Each node's set of itself and the nodes above it."""
    out = []
    for i, p in enumerate(parents):
        out.append({i} | (out[p] if 0 <= p < i else set()))
    return out


def words_of(nodes, words):
    w = np.zeros(words, dtype=np.uint32)
    for j in nodes:
        if j < 32 * words:
            w[j // 32] |= np.uint32(1 << (j % 32))
    return w.view(np.int32)


# ------------------------------------------------------------------------------ tree planning
def plan_tree_loops(parents, cu, seqlens_k, n_tok, words):
    mask, positions = np.zeros((n_tok, words), dtype=np.int32), np.full(n_tok, -1, dtype=np.int64)
    for b, n_k in enumerate(seqlens_k):
        t0 = min(max(cu[b], 0), n_tok)
        n = min(max(cu[b + 1], t0), n_tok) - t0
        for i, nodes in enumerate(ancestors(parents[t0:t0 + n])):
            mask[t0 + i] = words_of(nodes, words)
            positions[t0 + i] = max(n_k, 0) - n + len(nodes) - 1
    return mask, positions


@pytest.mark.parametrize("kind", ["tree", "chain", "star", "comb", "any"])
@pytest.mark.parametrize("sizes,words,pad", [
    ([1], 1, 0), ([2], 1, 3), ([31, 32, 33], 2, 0), ([8] * 8, 1, 5), ([0, 64, 0, 65, 1, 0], 3, 2), ([700], 22, 1),
    ([128, 1, 127, 96, 97], 4, 0), ([128, 1, 127, 96, 160, 161, 33], 5, 0), ([1100, 40], 40, 3), ([64, 40], 1, 0), ([200, 7], 3, 9), (None, 2, 40), ([], 1, 6), ([0, 0], 2, 4), ([30, 70], 9, 0),
])
def test_plan_tree_against_loops(kind, sizes, words, pad):
    rng = np.random.default_rng(words + pad)
    sizes = rng.integers(0, 65, 500).tolist() if sizes is None else sizes
    parents = [p for n in sizes for p in random_parents(rng, n, kind)] + [0] * pad
    cu = np.concatenate([[0], np.cumsum(sizes)]).astype(int).tolist()
    seqlens_k = [n + int(rng.integers(0, 5000)) for n in sizes]
    want = plan_tree_loops(parents, cu, seqlens_k, len(parents), words)
    args = (i32(parents), i32(cu), i32(seqlens_k), words)
    for _ in range(2):
        mask, positions = smla.sparse_mla_plan_tree(*args)
        assert np.array_equal(mask.cpu().numpy(), want[0]) and np.array_equal(positions.cpu().numpy(), want[1])


def test_plan_tree_clamps_sums_and_lengths():
    rng = np.random.default_rng(3)
    parents = random_parents(rng, 40, "any")
    for cu, lens in (([-5, 10, 1000], [3, 100]), ([4, 20, 30], [-9, 0]), ([7, 7, 7], [5, 5]), ([90, 95, 99], [1, 2])):
        mask, positions = smla.sparse_mla_plan_tree(i32(parents), i32(cu), i32(lens), 2)
        want = plan_tree_loops(parents, cu, lens, 40, 2)
        assert np.array_equal(mask.cpu().numpy(), want[0]) and np.array_equal(positions.cpu().numpy(), want[1])


def test_plan_tree_refuses_wrong_tensors():
    p, cu, k = i32([-1, 0, 0]), i32([0, 3]), i32([9])
    for kw in (dict(cu_seqlens_q=i32([0, 1, 3])), dict(mask_words=0), dict(mask_words=1025), dict(positions=i32([0, 0])),
               dict(tree_mask=i32([0, 0, 0])), dict(parents=i32([[-1, 0], [0, 0]])[:, 0]), dict(tree_mask=p.view(3, 1)), dict(positions=p)):
        with pytest.raises((ValueError, smla.SmlaError)):
            smla.sparse_mla_plan_tree(**dict(dict(parents=p, cu_seqlens_q=cu, seqlens_k=k, mask_words=1), **kw))


# ----------------------------------------------------------------------------- tree attention
def tree_case(seed, q_lens, k_lens, heads, d_qk=576, kind="tree", words=None, **kw):
    """chunk_case with a mask: ancestors of a random tree, or ("bits") any bits, later nodes' among them."""
    w, rng = chunk_case(seed, q_lens, k_lens, heads, d_qk, **kw), np.random.default_rng(seed)
    words = max(1, -(-max([*q_lens, 1]) // 32)) if words is None else words
    mask = rng.integers(-2 ** 31, 2 ** 31, (w["q"].shape[0], words))
    if kind != "bits":
        rows = [words_of(nodes, words) for n in q_lens for nodes in ancestors(random_parents(rng, n, kind))]
        mask[:len(rows)] = np.asarray(rows).reshape(-1, words)
    return dict(w, tree_mask=i32(mask))


def visible(w):
    """[n_tok, longest] truth values of what each token sees, from the definition."""
    cu, lens, mask = w["cu_seqlens_q"].tolist(), w["seqlens_k"].tolist(), w["tree_mask"].cpu().numpy().view(np.uint32)
    seen = np.zeros((w["q"].shape[0], max([*lens, 1])), dtype=bool)
    for b, n_k in enumerate(lens):
        before = max(n_k, 0) - (cu[b + 1] - cu[b])
        for t in range(cu[b], cu[b + 1]):
            seen[t, :max(before, 0)] = True
            bits = np.unpackbits(mask[t].view(np.uint8), bitorder="little").astype(bool)
            for j in range(max(-before, 0), min(cu[b + 1] - cu[b], len(bits))):
                seen[t, before + j] = bits[j]
    return torch.from_numpy(seen).cuda()


def tree_check(w, sink=None, sm_scale=None, run=None, **kw):
    """The operator against 64 bits, request by request, within the bound of its roundings."""
    q, cu, page = w["q"], w["cu_seqlens_q"].tolist(), w["page_block"]
    n, h, d = q.shape
    scale = d ** -0.5 if sm_scale is None else sm_scale
    mark = dict(out=torch.full((n, h, 512), 3.0, dtype=torch.bfloat16, device="cuda"),
                lse=torch.full((n, h), 5.0, device="cuda"), max_logits=torch.full((n, h), 7.0, device="cuda"))
    got = (run or smla.sparse_mla_tree_fwd_paged)(**w, attn_sink=sink, sm_scale=sm_scale, **mark, **kw)
    out, lse, top = got
    covered = torch.zeros(n, dtype=torch.bool, device="cuda")
    table, rows_total, sees = w["block_table"].long(), w["kv_pool"].shape[0], visible(w)
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
            seen = ok[None, :] & sees[a:e, :n_k]
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
def test_tree_heads(heads, d_qk):
    tree_check(tree_case(heads, [1, 3, 10], [77, 3, 200], heads, d_qk))
    tree_check(tree_case(heads + 1, [12, 5], [333, 64], heads, d_qk, kind="bits"))


@pytest.mark.parametrize("page", [1, 7, 8, 16, 24, 32, 64, 100, 256])
def test_tree_pages(page):
    tree_check(tree_case(page, [2, 9, 1], [130, 65, 300], 16, page=page))
    tree_check(tree_case(page + 1, [5, 40], [64, 129], 128, 512, kind="bits", page=page))


@pytest.mark.parametrize("n_q", [1, 2, 8, 16, 31, 32, 33, 63, 64, 65, 100])
@pytest.mark.parametrize("before", [0, 1, 31, 32, 33, 63, 64, 95, 127, 500])
def test_tree_sizes(n_q, before):
    """The new keys begin and end anywhere in a block of 64 keys, and in the words of the mask."""
    tree_check(tree_case(n_q + before, [n_q], [n_q + before], 32, kind="bits"))
    tree_check(tree_case(n_q, [n_q], [n_q + before], 128, 512))


@pytest.mark.parametrize("sink", [True, False])
@pytest.mark.parametrize("kind", ["tree", "star", "chain", "bits"])
@pytest.mark.parametrize("heads,d_qk", [(16, 576), (20, 512), (128, 576), (200, 576)])
def test_tree_ragged(kind, sink, heads, d_qk):
    w = tree_case(heads, [0, 17, 1, 0, 64, 5, 130], [40, 17, 900, 0, 333, 5, 200], heads, d_qk, kind, tail=3)
    tree_check(w, torch.randn(heads, device="cuda") * 3 if sink else None)


def test_tree_mask_words():
    """Fewer words than nodes (the nodes behind them are seen by none), and more."""
    for words in (1, 2, 3, 7):
        for kind in ("tree", "bits"):
            tree_check(tree_case(words, [70, 3, 40], [200, 50, 40], 24, kind=kind, words=words))


def test_tree_rows_that_see_nothing():
    # no cached keys and an empty mask; more nodes than keys; no keys at all; a negative length; an ordinary request
    w = tree_case(3, [4, 9, 4, 2, 6], [4, 5, 0, 0, 50], 48)
    w["seqlens_k"][3] = -3
    w["tree_mask"][:3] = 0
    for sink in (None, torch.randn(48, device="cuda")):
        tree_check(w, sink)
    w["tree_mask"][:] = 0
    tree_check(w)
    w["tree_mask"][:] = -1
    tree_check(w)


@pytest.mark.parametrize("heads", [16, 128])
def test_tree_unmapped_pages(heads):
    w = tree_case(6, [4, 3, 30], [400, 500, 130], heads, page=16)
    w["block_table"][0, 3] = -1
    w["block_table"][0, 20:] = -7
    w["block_table"][1, :] = 2 ** 30           # past the pool
    w["block_table"][2, 1] = w["kv_pool"].shape[0] // 16
    w["block_table"][2, 8] = -1                # the nodes' own last page
    tree_check(w)
    tree_check(tree_case(7, [4, 20], [300, 20], 32, page=16, width=10))    # a table shorter than the keys


def test_tree_large_scores_and_sinks():
    tree_check(tree_case(8, [3, 40], [700, 650], 16, scale=12.0))
    tree_check(tree_case(9, [2], [2000], 128, scale=0.01), sm_scale=3.0)
    tree_check(tree_case(4, [3, 1], [70, 9], 6), torch.tensor([float("-inf"), -100.0, -1.0, 0.0, 30.0, 80.0], device="cuda"))


@pytest.mark.parametrize("shape", [([8] * 40, [50 + 77 * i for i in range(40)], 128), ([7], [20000], 128), ([5], [20000], 16),
                                   ([3, 1, 61], [9000, 11, 5000], 128), ([300], [1500], 64), ([2] * 500, [90] * 500, 20)])
def test_tree_splits_and_joins(shape):
    """Sizes where requests are cut over workers and joined, evenly and not."""
    q_lens, k_lens, heads = shape
    tree_check(tree_case(len(q_lens), q_lens, k_lens, heads))


def test_tree_causal_masks_are_the_causal_form():
    """The same set of keys: each side is within its own bound of the same values."""
    for heads in (16, 128):
        w = tree_case(heads, [9, 64, 1], [700, 64, 300], heads, kind="chain")
        out, lse, top = tree_check(w)
        w.pop("tree_mask")
        o2, l2, t2 = smla.sparse_mla_chunk_fwd_paged(**w)
        assert torch.equal(top, t2) and float((lse - l2).abs().max()) <= 1e-4
        assert float((out.float() - o2.float()).norm()) <= 2 * 1.5 * U16 * float(o2.float().norm())


def test_tree_full_masks_are_the_form_without_causality():
    """Random shapes, from one worker's to all workers' at once: the same set of keys, cut and joined another way."""
    rng = np.random.default_rng(11)
    for i in range(40):
        heads, page = int(rng.choice([1, 8, 16, 20, 64, 128, 160, 512])), int(rng.choice([16, 32, 64]))
        n_req = int(rng.choice([1, 2, 5, 33, 80]))
        q_lens = rng.integers(0, int(rng.choice([2, 9, 33])) + 1, n_req).tolist()
        k_lens = [q + int(10 ** rng.uniform(0, 3.6 if n_req > 5 else 4.2)) for q in q_lens]
        while sum(q_lens) * heads > 60000:
            q_lens = [q // 2 for q in q_lens]
        w = chunk_case(i, q_lens, k_lens, heads, int(rng.choice([512, 576])), page=page, tail=1)
        sink = torch.randn(heads, device="cuda") if i % 3 == 0 else None
        n = sum(q_lens)
        mask = torch.full((n + 1, max(1, -(-max([*q_lens, 1]) // 32))), -1, dtype=torch.int32, device="cuda")
        a = smla.sparse_mla_tree_fwd_paged(**w, tree_mask=mask, attn_sink=sink)
        b = smla.sparse_mla_chunk_fwd_paged(**w, causal=False, attn_sink=sink)
        if n:
            # the scores are the same; the sums' order and the exponents' offsets are not
            assert torch.equal(a[2][:n], b[2][:n]) and float((a[1][:n] - b[1][:n]).abs().max()) <= 1e-4, i
            assert float((a[0][:n].float() - b[0][:n].float()).norm()) <= 2 * 1.5 * U16 * float(b[0][:n].float().norm()), i


def test_tree_pool_past_2_gib():
    rows = 2_500_032
    pool = torch.empty(rows, 1, 576, device="cuda", dtype=torch.bfloat16).normal_()
    table = i32(np.array([[rows // 64 - 1, 3, rows // 64 - 2, 39000, 20]]))
    tree_check(dict(q=torch.randn(5, 128, 576, device="cuda").to(torch.bfloat16), kv_pool=pool, block_table=table,
                    cu_seqlens_q=i32([0, 5]), seqlens_k=i32([300]), page_block=64, tree_mask=i32([[1], [3], [5], [11], [21]])))


def test_tree_twice_the_same_bits_streams_and_threads():
    w = tree_case(14, [1, 60, 2, 9], [5000, 400, 3001, 700], 128)
    want = smla.sparse_mla_tree_fwd_paged(**w)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    many = [smla.sparse_mla_tree_fwd_paged(**w, stream=s) for _ in range(4) for s in streams]
    same = []

    def work():
        s = torch.cuda.Stream()
        got = [smla.sparse_mla_tree_fwd_paged(**w, stream=s) for _ in range(10)]
        s.synchronize()
        same.append(all(torch.equal(x, y) for g in got for x, y in zip(want, g)))

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert same == [True] * 3 and all(torch.equal(x, y) for g in many for x, y in zip(want, g))


def test_tree_in_graphs_with_changing_masks_and_lengths():
    """Two captured calls with a workspace each, replayed after masks and lengths changed in place."""
    ws = [tree_case(16 + i, [8, 20], [900, 600], 128) for i in range(2)]
    graphs, outs = [], []
    for w in ws:
        smla.sparse_mla_tree_fwd_paged(**w)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(smla.sparse_mla_tree_fwd_paged(**w))
        graphs.append(g)
    rng = np.random.default_rng(0)
    for lens, cu in (([900, 600], [0, 8, 28]), ([40, 333], [0, 1, 28]), ([900, 20], [0, 20, 28]), ([0, 600], [0, 0, 28])):
        for w in ws:
            w["seqlens_k"].copy_(i32(lens))
            w["cu_seqlens_q"].copy_(i32(cu))
            w["tree_mask"].copy_(i32(rng.integers(-2 ** 31, 2 ** 31, (28, 1))))
        for g in graphs:
            g.replay()
        for w, o in zip(ws, outs):
            tree_check(w, run=lambda o=o, **kw: [dst.copy_(src) for dst, src in zip((kw["out"], kw["lse"], kw["max_logits"]), o)])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_tree_broken_queries_stay_visible(bad):
    for q_lens, k_lens, heads, d_qk in (([3], [70], 4, 576), ([5, 1], [700, 5000], 128, 512)):
        w = tree_case(heads, q_lens, k_lens, heads, d_qk)
        want = smla.sparse_mla_tree_fwd_paged(**w)
        broken = torch.zeros(w["q"].shape[:2], dtype=torch.bool, device="cuda")
        broken[0, 1] = broken[-1, heads - 1] = True
        w["q"][..., 5] = torch.where(broken, bad, w["q"][..., 5])
        got = smla.sparse_mla_tree_fwd_paged(**w)
        for g, x in zip(got, want):
            assert bool(g[broken].isnan().all()) and torch.equal(g[~broken], x[~broken])


def test_tree_nan_keys_reach_the_tokens_that_see_them_and_no_other_request():
    for n_k, heads in ((100, 16), (9000, 128)):
        w = tree_case(22, [4, 2, 5], [n_k, 90, 300], heads)
        w["tree_mask"][:4] = i32([[1], [3], [5], [9]])            # the first request: three children of its first node
        at = n_k - 3                                              # the second node's position
        w["kv_pool"][w["block_table"][0, at // 64].long() * 64 + at % 64, 0, 7] = float("nan")
        out, lse, top = smla.sparse_mla_tree_fwd_paged(**w)
        assert bool(lse[1].isnan().all()) and bool(top[1].isnan().all()) and bool(out[1].isnan().any(-1).all())
        # its siblings do not see it: their scores and sums are whole, and so is everything of the other requests
        assert bool(torch.isfinite(lse[[0, 2, 3]]).all()) and bool(torch.isfinite(top[[0, 2, 3]]).all())
        assert all(bool(torch.isfinite(x[4:].float()).all()) for x in (out, lse, top))


def test_tree_refuses_wrong_tensors():
    w = tree_case(18, [2], [70], 16)
    for kw in (dict(tree_mask=w["tree_mask"][:1]), dict(tree_mask=w["tree_mask"][:, 0]), dict(tree_mask=w["tree_mask"].long()),
               dict(tree_mask=w["tree_mask"].cpu()), dict(tree_mask=torch.zeros(2, 0, dtype=torch.int32, device="cuda")),
               dict(tree_mask=torch.zeros(2, 1025, dtype=torch.int32, device="cuda")), dict(seqlens_k=i32([1, 2])),
               dict(kv_pool=w["kv_pool"][..., :512].contiguous()), dict(attn_sink=torch.zeros(3, device="cuda")),
               dict(d_v=256), dict(sm_scale=-1.0), dict(page_block=0), dict(lse=w["tree_mask"].view(torch.float32))):
        with pytest.raises((ValueError, TypeError, smla.SmlaError)):
            smla.sparse_mla_tree_fwd_paged(**dict(w, **kw))


# ------------------------------------------------------------------------------- verification
def verify_loops(target, draft, tokens, parents, cu, accept_u, sample_u, max_keep):
    """The rule as the header states it: rows in fp32, sums and comparisons in 64 bits."""
    n_tok, vocab = target.shape
    target = np.where(target > 0, target, np.float32(0))
    keep, out = (np.full((len(sample_u), max_keep), -1) for _ in range(2))
    n_keep = []
    for b in range(len(sample_u)):
        t0 = min(max(cu[b], 0), n_tok)
        n = min(min(max(cu[b + 1], t0), n_tok) - t0, 1024)
        if n == 0:
            n_keep.append(0)
            continue
        cur, kept, path, said = 0, 1, [0], []
        while True:
            p, C, Z = target[t0 + cur], np.float32(0), 1.0
            q = None if draft is None else draft[t0 + cur].astype(np.float64)
            r, chosen = p.copy(), None
            for c in range(cur + 1, n):
                if parents[t0 + c] != cur or kept >= max_keep or not 0 <= tokens[t0 + c] < vocab:
                    continue
                x = tokens[t0 + c]
                if float(accept_u[t0 + c]) * (1.0 if q is None else q[x]) * Z < float(r[x]):
                    chosen = c
                    break
                if q is None:
                    Z -= float(r[x])
                    r[x] = 0
                else:
                    C = np.float32(float(C) + Z)
                    r = np.maximum(p.astype(np.float64) - float(C) * q, 0).astype(np.float32)
                    Z = float(r.astype(np.float64).sum())
            if chosen is None:
                break
            cur, kept = chosen, kept + 1
            path.append(cur)
            said.append(tokens[t0 + cur])
        if not r.any():
            r = p
        sums = r.astype(np.float64).cumsum()
        over = np.flatnonzero(sums > max(float(sample_u[b]), 0.0) * sums[-1])
        some = np.flatnonzero(r)
        said.append(min(over[0], some[-1]) if len(over) else some[-1] if len(some) else -1)
        keep[b, :kept], out[b, :kept] = path, said
        n_keep.append(kept)
    return keep, out, np.asarray(n_keep)


def verify_case(seed, sizes, vocab, draft=True, kind="tree", scale=2.0, apart=1.0, pad=0, sharp=False):
    """Trees whose tokens are drawn from the draft's rows (or, without a draft, chosen among the likely ones)."""
    g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    n = int(sum(sizes)) + pad
    logits = torch.randn(n, vocab, generator=g) * scale
    near = logits + torch.randn(n, vocab, generator=g) * apart
    target, q = logits.softmax(-1), near.softmax(-1)
    cu = np.concatenate([[0], np.cumsum(sizes)]).astype(int).tolist()
    parents = [p for m in sizes for p in random_parents(rng, m, kind)] + [0] * pad
    tokens = np.zeros(n, dtype=np.int64)
    for b, m in enumerate(sizes):
        for i in range(1, m):
            p = parents[cu[b] + i]
            row = q[cu[b] + (p if 0 <= p < i else 0)]
            tokens[cu[b] + i] = int(torch.multinomial(row, 1, generator=g)) if draft else int(row.topk(min(vocab, 1 + i % 3)).indices[-1])
    return dict(target_probs=target.cuda(), draft_probs=q.cuda() if draft else None, tokens=i32(tokens), parents=i32(parents),
                cu_seqlens_q=i32(cu), accept_u=torch.rand(n, generator=g).cuda(), sample_u=torch.rand(len(sizes), generator=g).cuda(),
                max_keep=max([*sizes, 1]))


def verify_check(w, **kw):
    def host(x):
        return None if x is None else x.cpu().numpy()
    want = verify_loops(host(w["target_probs"]), host(w["draft_probs"]), host(w["tokens"]).astype(np.int64),
                        host(w["parents"]).astype(np.int64), w["cu_seqlens_q"].tolist(), host(w["accept_u"]), host(w["sample_u"]),
                        w["max_keep"])
    got = smla.sparse_mla_verify_tree(**w, **kw)
    for g, x, name in zip(got, want, ("keep", "out_tokens", "n_keep")):
        assert np.array_equal(g.cpu().numpy(), x), name
    return got


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 32, 33, 255, 256, 257, 1000, 4095, 16385, 50001])
def test_verify_vocabularies(vocab, draft):
    for kind in ("chain", "tree", "star"):
        verify_check(verify_case(vocab, [6, 1, 4, 9], vocab, draft, kind))


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("kind", ["chain", "tree", "star", "any"])
def test_verify_many_requests(draft, kind):
    rng = np.random.default_rng(1)
    for apart in (0.1, 1.0, 4.0):
        w = verify_case(int(apart * 10), rng.integers(0, 14, 300).tolist(), 97, draft, kind, apart=apart, pad=4)
        kept = verify_check(w)[2]
        for m in (1, 2, 3):
            verify_check(dict(w, max_keep=m))
    assert int(kept.max()) > 1


def test_verify_large_vocabulary():
    verify_check(verify_case(5, [4, 3, 7], 151_643, kind="star", apart=2.0))
    verify_check(verify_case(6, [4, 3, 7], 128_000, False, "star"))
    for vocab in (5_000_003, 3_000_000):
        verify_check(verify_case(7, [3, 2], vocab, vocab % 2 == 1, "star", scale=0.5))


def test_verify_rows_far_apart():
    """Strided rows, and rows past 2^31 elements."""
    w = verify_case(7, [5, 3], 1000)
    wide = torch.zeros(8, 1300, device="cuda")
    wide[:, 7:1007] = w["target_probs"]
    draft = torch.zeros(8, 1001, device="cuda")
    draft[:, 1:] = w["draft_probs"]
    got = verify_check(dict(w, target_probs=wide[:, 7:1007], draft_probs=draft[:, 1:]))
    assert all(torch.equal(a, b) for a, b in zip(got, smla.sparse_mla_verify_tree(**w)))
    far = torch.empty(2_600_000_000, device="cuda")[:8 * 325_000_000].view(8, 325_000_000)[:, :1000]
    far.copy_(w["target_probs"])
    got2 = smla.sparse_mla_verify_tree(**dict(w, target_probs=far, draft_probs=far.clone()))
    verify_check(dict(w, draft_probs=w["target_probs"]))
    assert all(torch.equal(a, b) for a, b in zip(got2, smla.sparse_mla_verify_tree(**dict(w, draft_probs=w["target_probs"]))))


def test_verify_random_numbers_at_their_ends():
    for draft in (True, False):
        w = verify_case(8, [5, 1, 9, 3], 300, draft, "star")
        w["target_probs"][:, :3] = 0.0
        w["target_probs"][:, -2:] = 0.0
        for a in (0.0, 1.0 - 2.0 ** -24):
            for s in (0.0, 1.0 - 2.0 ** -24, 1.0, 3.0, -1.0):
                w["accept_u"].fill_(a)
                w["sample_u"].fill_(s)
                verify_check(w)
        w["sample_u"].fill_(float("nan"))       # counts as 0
        got = smla.sparse_mla_verify_tree(**w)
        w["sample_u"].fill_(0.0)
        assert all(torch.equal(a, b) for a, b in zip(got, smla.sparse_mla_verify_tree(**w)))


def test_verify_probabilities_at_their_ends():
    # the draft is the target: a drafted token is always kept
    w = verify_case(9, [6, 6], 500, kind="chain", apart=0.0)
    w["draft_probs"] = w["target_probs"]
    assert verify_check(w)[2].tolist() == [6, 6]
    # one token has everything; it was drafted, or it was not
    w = verify_case(10, [4] * 6, 40, kind="star")
    w["target_probs"].zero_()
    w["target_probs"][:, 17] = 1.0
    for draft in (w["draft_probs"], None):
        for x in (17, 18):
            w["tokens"].fill_(x)
            out = verify_check(dict(w, draft_probs=draft))[1]
            assert bool((out[:, 0] == 17).all())
    # twice the same child; tokens that the draft's row says are impossible
    w = verify_case(11, [7] * 20, 12, kind="star")
    w["tokens"].fill_(3)
    for draft in (w["draft_probs"], None, torch.zeros_like(w["draft_probs"])):
        verify_check(dict(w, draft_probs=draft))
    # nothing is left behind a rejection: the target's own row
    w = verify_case(12, [3] * 20, 30, kind="star")
    w["draft_probs"] = w["target_probs"] * 2
    w["accept_u"].fill_(0.9)
    verify_check(w)


def test_verify_nan_negative_and_empty_rows():
    for draft in (True, False):
        w = verify_case(13, [5, 4, 1, 6], 200, draft, "star")
        p = w["target_probs"]
        p[:, ::7] = float("nan")
        p[:, 1::7] = -0.5
        verify_check(w)
        p[:5] = 0.0
        p[5:9] = float("nan")
        out = verify_check(w)[1]
        assert out[0, 0] == -1 and out[1, 0] == -1 and out[2, 0] >= 0


def test_verify_tokens_and_parents_out_of_range():
    for draft in (True, False):
        w = verify_case(14, [9] * 30, 50, draft, "any")
        rng = np.random.default_rng(2)
        bad = rng.choice([-1, 50, 2 ** 31 - 1, -2 ** 31], 270)
        w["tokens"] = torch.where(i32(rng.integers(0, 3, 270)) == 0, i32(bad), w["tokens"])
        verify_check(w)
        for cu in ([-5, 9, 2000], [3, 2, 40], [300, 400, 500], [5, 5, 5]):
            verify_check(dict(w, cu_seqlens_q=i32(cu), sample_u=w["sample_u"][:2].contiguous()))


def test_verify_large_trees():
    for kind, n in (("chain", 100), ("star", 700), ("tree", 1024), ("star", 1500), ("chain", 1300)):
        w = verify_case(n, [n, 3], 64, kind=kind, apart=0.05)
        verify_check(w)
        verify_check(dict(w, draft_probs=None))
    w = verify_case(15, [1100], 8, kind="star")
    w["accept_u"].fill_(1.0 - 2.0 ** -24)
    w["tokens"].copy_(w["target_probs"][0].argmin())
    verify_check(dict(w, draft_probs=None))
    verify_check(w)


@pytest.mark.parametrize("draft", [True, False])
def test_verify_follows_the_target(draft):
    """20000 requests with one distribution: whatever is drafted, the first token out is distributed as the target's, and
    the second behind each first one.  Counts of independent draws: within five standard deviations."""
    n_req, vocab, sizes = 20000, 6, 4
    g = torch.Generator(device="cuda").manual_seed(16)
    p = torch.tensor([[0.4, 0.3, 0.15, 0.1, 0.05, 0.0], [0.1, 0.1, 0.2, 0.2, 0.2, 0.2]], device="cuda")
    q = torch.tensor([0.1, 0.2, 0.4, 0.1, 0.1, 0.1], device="cuda")
    # node 0's children are 1 and 2, node 3 is behind node 1; every node but 0 has the second row behind it
    target = p[torch.tensor([0, 1, 1, 1], device="cuda")].repeat(n_req, 1)
    tokens = torch.multinomial(q.expand(n_req * sizes, -1), 1, generator=g).squeeze(1).to(torch.int32).view(n_req, sizes)
    if not draft:        # chosen outright: 2 and 1 first
        tokens[:, 1:3] = i32([2, 1])
    kw = dict(target_probs=target, tokens=tokens.flatten(), parents=i32([-1, 0, 0, 1]).repeat(n_req),
              cu_seqlens_q=torch.arange(n_req + 1, device="cuda", dtype=torch.int32) * sizes,
              accept_u=torch.rand(n_req * sizes, generator=g, device="cuda"), sample_u=torch.rand(n_req, generator=g, device="cuda"))
    keep, out, n_keep = smla.sparse_mla_verify_tree(**kw, max_keep=3, draft_probs=q.expand(n_req * sizes, -1).contiguous() if draft else None)
    first = torch.bincount(out[:, 0].long(), minlength=vocab).double()
    want = p[0].double() * n_req
    assert bool(((first - want).abs() <= 5 * (want * (1 - p[0].double())).sqrt()).all())
    second = out[n_keep > 1, 1].long()
    total = second.numel()
    assert total > 2000
    want = p[1].double() * total
    assert bool(((torch.bincount(second, minlength=vocab).double() - want).abs() <= 5 * (want * (1 - p[1].double())).sqrt()).all())


def test_verify_streams_threads_and_graphs():
    w = verify_case(17, [5, 9, 1, 3] * 10, 5000)
    want = verify_check(w)
    torch.cuda.synchronize()
    streams, same = [torch.cuda.Stream() for _ in range(3)], []
    many = [smla.sparse_mla_verify_tree(**w, stream=s) for _ in range(4) for s in streams]

    def work():
        s = torch.cuda.Stream()
        got = [smla.sparse_mla_verify_tree(**w, stream=s) for _ in range(10)]
        s.synchronize()
        same.append(all(torch.equal(x, y) for g in got for x, y in zip(want, g)))

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert same == [True] * 3 and all(torch.equal(x, y) for g in many for x, y in zip(want, g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = smla.sparse_mla_verify_tree(**w)
    for _ in range(3):
        w["accept_u"].copy_(torch.rand_like(w["accept_u"]))
        w["sample_u"].copy_(torch.rand_like(w["sample_u"]))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(captured, verify_check(w)))


def test_verify_refuses_wrong_tensors():
    w = verify_case(18, [4, 3], 50)
    p = w["target_probs"]
    for kw in (dict(target_probs=p.half()), dict(target_probs=p[:3]), dict(target_probs=p[0]), dict(target_probs=p[:, ::2]),
               dict(draft_probs=p[:, :49]), dict(draft_probs=p.double()), dict(tokens=w["tokens"][:3]), dict(parents=w["parents"][:3]),
               dict(accept_u=w["accept_u"][:3]), dict(sample_u=w["sample_u"][:1]), dict(max_keep=0), dict(target_probs=p.cpu()),
               dict(keep=i32([[0, 0]])), dict(n_keep=i32([0, 0, 0])), dict(keep=w["tokens"][:2].view(2, 1), max_keep=1),
               dict(target_probs=p[:1].expand(7, -1))):
        with pytest.raises((ValueError, TypeError, smla.SmlaError)):
            smla.sparse_mla_verify_tree(**dict(w, **kw))


def test_verify_of_no_requests_and_no_nodes():
    w = verify_case(19, [0, 0], 20, pad=2)
    keep, out, n_keep = smla.sparse_mla_verify_tree(**w)
    assert keep.tolist() == [[-1], [-1]] and out.tolist() == [[-1], [-1]] and n_keep.tolist() == [0, 0]
    empty = dict(w, **{k: w[k][:0] for k in ("target_probs", "draft_probs", "tokens", "parents", "accept_u")})
    assert [x.tolist() for x in smla.sparse_mla_verify_tree(**empty)] == [[[-1], [-1]], [[-1], [-1]], [0, 0]]
    none = smla.sparse_mla_verify_tree(**dict(w, cu_seqlens_q=i32([0]), sample_u=w["sample_u"][:0]))
    assert [tuple(x.shape) for x in none] == [(0, 1), (0, 1), (0,)]


# ------------------------------------------------------------------------------------- commit
def commit_loops(keep, n_keep, cu, seqlens_k, table, pool, page, free, start):
    """pool [layers, rows, d]; returns lengths, counts; changes pool and free."""
    rows_total, width = pool.shape[1], table.shape[1]

    def row(b, pos):
        if pos < 0 or pos // page >= width or table[b, pos // page] < 0:
            return -1
        r = int(table[b, pos // page]) * page + pos % page
        return r if r < rows_total else -1

    lengths, at, lost, kept = [], start, 0, 0
    for b, n_k in enumerate(seqlens_k):
        n_k, fresh = max(n_k, 0), max(cu[b + 1] - cu[b], 0)
        before = n_k - fresh
        m = min(n_keep[b], fresh, keep.shape[1])
        for i in range(max(m, 0)):
            if i < keep[b, i] < fresh:
                src, dst = row(b, before + int(keep[b, i])), row(b, before + i)
                if src >= 0 and dst >= 0:
                    pool[:, dst] = pool[:, src]
        kept += max(m, 0)
        lengths.append(0 if n_keep[b] < 0 else max(before + m, 0))
        if free is not None and len(free):
            for col in range(min(-(-lengths[-1] // page), width), min(-(-n_k // page), width)):
                if table[b, col] >= 0:
                    if at > 0:
                        at -= 1
                        free[at] = table[b, col]
                    else:
                        lost += 1
    return lengths, [kept, at, lost]


def commit_case(seed, sizes, page, layers, d_qk=576, old_max=100, most=9, done=0.1, holes=0.0):
    rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    n_req = len(sizes)
    old = rng.integers(0, old_max + 1, n_req)
    width = -(-(old_max + max([*sizes, 1])) // page) + 1
    held = [-(-int(o + m) // page) for o, m in zip(old, sizes)]
    n_pages = sum(held) + 4
    pages = rng.permutation(n_pages)
    table, at = np.full((n_req, width), -1), 0
    for b, h in enumerate(held):
        table[b, :h] = pages[at:at + h]
        at += h
    table[rng.random(table.shape) < holes] = -1
    keep, n_keep = np.full((n_req, most), -1), np.zeros(n_req, dtype=int)
    for b, m in enumerate(sizes):
        k = int(rng.integers(0, min(m, most) + 1))
        keep[b, :k] = sorted(rng.choice(m, k, replace=False)) if k else []
        n_keep[b] = -1 if rng.random() < done else k
    shape = (layers, n_pages * page, 1, d_qk) if layers else (n_pages * page, 1, d_qk)
    return dict(keep=i32(keep), n_keep=i32(n_keep), cu_seqlens_q=i32(np.concatenate([[0], np.cumsum(sizes)])),
                seqlens_k=i32(old + np.asarray(sizes, dtype=int)), block_table=i32(table),
                kv_pool=torch.randn(shape, generator=g).to(torch.bfloat16).cuda(), page_block=page,
                free_pages=i32(np.concatenate([np.full(at, -5), pages[at:]])), free_start=i32([at]))


def commit_check(w):
    pool = None if w["kv_pool"] is None else w["kv_pool"].reshape(-1, w["kv_pool"].shape[-3], w["kv_pool"].shape[-1]).clone()
    free = None if w["free_pages"] is None else w["free_pages"].cpu().numpy().copy()
    start = 0 if free is None else len(free) if w["free_start"] is None else min(max(int(w["free_start"]), 0), len(free))
    host = [w[k].cpu().numpy().astype(np.int64) for k in ("keep", "n_keep", "cu_seqlens_q", "seqlens_k", "block_table")]
    lengths, counts = commit_loops(*host, torch.zeros(1, 0, 512) if pool is None else pool, w["page_block"], free, start)
    untouched = [w[k].clone() for k in ("keep", "n_keep", "cu_seqlens_q", "seqlens_k", "block_table")]
    got = smla.sparse_mla_commit_tree(**w)
    assert got[0].tolist() == lengths and got[1].tolist() == counts
    if pool is not None:
        assert torch.equal(w["kv_pool"].reshape(pool.shape).view(torch.int16), pool.view(torch.int16))
    if free is not None:
        assert np.array_equal(w["free_pages"].cpu().numpy(), free)
    assert all(torch.equal(a, w[k]) for a, k in zip(untouched, ("keep", "n_keep", "cu_seqlens_q", "seqlens_k", "block_table")))
    return got


@pytest.mark.parametrize("page", [1, 7, 16, 64, 100])
@pytest.mark.parametrize("layers,d_qk", [(0, 576), (1, 512), (3, 576), (5, 512)])
def test_commit_against_loops(page, layers, d_qk):
    rng = np.random.default_rng(page)
    commit_check(commit_case(page, rng.integers(0, 33, 20).tolist(), page, layers, d_qk))
    commit_check(commit_case(page + 1, [8], page, layers, d_qk, done=0))
    commit_check(commit_case(page + 2, [70, 3, 64], page, layers, d_qk, most=70, done=0, holes=0.1))


@pytest.mark.parametrize("n_req", [0, 1, 255, 256, 257, 700])
def test_commit_many_requests(n_req):
    rng = np.random.default_rng(n_req)
    commit_check(commit_case(n_req, rng.integers(0, 12, n_req).tolist(), 16, 2, 512))
    commit_check(commit_case(n_req, rng.integers(0, 3, n_req).tolist(), 4, 1, 576, old_max=400, done=0.5))


def test_commit_long_requests_that_are_done():
    """Requests with many pages, ended beside ones that go on; holes in their tables."""
    rng = np.random.default_rng(0)
    for n_req, old_max, page, holes in ((5, 3000, 4, 0.0), (70, 400, 1, 0.2), (300, 900, 8, 0.05), (33, 5 * 16, 16, 0.0)):
        commit_check(commit_case(n_req, rng.integers(0, 9, n_req).tolist(), page, 1, 512, old_max=old_max, done=0.4, holes=holes))


def test_commit_counts_of_every_kind():
    """More kept than there are nodes or entries, none, done; entries that do not ascend or lie outside stay inside
    the request's own new rows."""
    w = commit_case(3, [6, 6, 6, 6, 0, 2], 4, 2, done=0)
    w["n_keep"].copy_(i32([100, 6, 0, -1, 3, 9]))
    w["keep"][0] = torch.arange(9, device="cuda")
    w["keep"][1] = i32([0, 1, 3, 4, 5, -1, -1, -1, -1])
    commit_check(w)
    w = commit_case(4, [6, 6, 6], 4, 2, done=0)
    before = w["kv_pool"].clone()
    w["n_keep"].fill_(6)
    w["keep"].copy_(i32([[5, 4, 3, 2, 1, 0, 0, 0, 0], [2 ** 31 - 1, -2 ** 31, 6, 7, -1, 9, 0, 0, 0], [5] * 9]))
    smla.sparse_mla_commit_tree(**w)
    new = torch.zeros(before.shape[1], dtype=torch.bool, device="cuda")
    for b in range(3):
        for pos in range(int(w["seqlens_k"][b]) - 6, int(w["seqlens_k"][b])):
            new[int(w["block_table"][b, pos // 4]) * 4 + pos % 4] = True
    assert torch.equal(w["kv_pool"][:, ~new], before[:, ~new])
    assert torch.equal(w["kv_pool"][:, new][..., :1].sort(1).values.isnan(), before[:, new][..., :1].sort(1).values.isnan())


def test_commit_lengths_that_do_not_fit():
    w = commit_case(5, [6, 6, 6], 4, 1, done=0)
    w["seqlens_k"].copy_(i32([3, -4, 2 ** 31 - 1]))     # more nodes than keys, a negative length, keys past the table
    commit_check(w)
    w["cu_seqlens_q"].copy_(i32([0, 6, 2, 8]))
    commit_check(w)
    w = commit_case(6, [5, 5], 4, 1, done=0)
    w["block_table"][0] = 2 ** 30                       # past the pool: rows stay, the entries go back all the same
    commit_check(w)


def test_commit_free_list_ends():
    for start in (0, 1, 3, -2, 10 ** 6, None):
        w = commit_case(7, [9] * 12, 2, 1, done=0.5)
        w["free_start"] = None if start is None else i32([start])
        commit_check(w)
    w = commit_case(8, [9] * 12, 2, 1)
    commit_check(dict(w, free_pages=None, free_start=None))
    commit_check(dict(w, free_pages=w["free_pages"][:0]))
    commit_check(dict(w, kv_pool=None))


def test_commit_layers_apart_and_rows_past_2_gib():
    w = commit_case(9, [20, 31, 7], 16, 3, done=0)
    rows = w["kv_pool"].shape[1]
    wide = torch.full((3, rows + 48, 1, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :rows] = w["kv_pool"]
    commit_check(w)
    smla.sparse_mla_commit_tree(**dict(w, kv_pool=wide[:, :rows], free_pages=None, free_start=None))
    assert torch.equal(wide[:, :rows], w["kv_pool"]) and bool((wide[:, rows:] == 7).all())
    pool = torch.zeros(2, 1_500_000, 1, 576, dtype=torch.bfloat16, device="cuda")
    table = i32([[1_500_000 // 16 - 1, 1_400_000 // 16]])
    at = [int(table[0, x // 16]) * 16 + x % 16 for x in range(32)]
    pool[:, at] = torch.randn(2, 32, 1, 576, device="cuda").to(torch.bfloat16)
    before = pool[:, at].clone()
    smla.sparse_mla_commit_tree(i32([[0, 5, 20, 27]]), i32([4]), i32([0, 28]), i32([32]), table, pool, page_block=16)
    assert torch.equal(pool[:, at[4:8]], before[:, [4, 9, 24, 31]]) and int((pool != 0).any(-1).sum()) == 64


def test_commit_nan_bits_are_copied():
    w = commit_case(10, [12, 9], 4, 2, done=0)
    bits = torch.randint(-2 ** 15, 2 ** 15, w["kv_pool"].shape, device="cuda").to(torch.int16)
    w["kv_pool"] = bits.view(torch.bfloat16)
    commit_check(w)


def test_commit_streams_and_graphs():
    ws = [commit_case(11 + i, [9, 20, 3, 31], 8, 4) for i in range(3)]
    streams = [torch.cuda.Stream() for _ in ws]
    want = [{k: v.clone() if torch.is_tensor(v) else v for k, v in w.items()} for w in ws]
    want_out = [smla.sparse_mla_commit_tree(**w) for w in want]
    torch.cuda.synchronize()
    got = [smla.sparse_mla_commit_tree(**w, stream=s) for w, s in zip(ws, streams)]
    torch.cuda.synchronize()
    for w, x, g, o in zip(ws, want, got, want_out):
        assert all(torch.equal(a, b) for a, b in zip(g, o)) and torch.equal(w["kv_pool"], x["kv_pool"])
    w = commit_case(20, [9, 20, 3, 31], 8, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = smla.sparse_mla_commit_tree(**w)
    for seed in (21, 22):
        x = commit_case(seed, [9, 20, 3, 31], 8, 4)
        for k in ("keep", "n_keep", "seqlens_k", "block_table", "free_start"):
            w[k].copy_(x[k])
        w["block_table"].clamp_(max=(w["kv_pool"].shape[1] // 8) - 1)
        y = {k: v.clone() if torch.is_tensor(v) else v for k, v in w.items()}
        graph.replay()
        out = smla.sparse_mla_commit_tree(**y)
        assert all(torch.equal(a, b) for a, b in zip(captured, out))
        assert torch.equal(w["kv_pool"], y["kv_pool"]) and torch.equal(w["free_pages"], y["free_pages"])


def test_commit_refuses_wrong_tensors():
    w = commit_case(12, [4, 3], 4, 2)
    pool = w["kv_pool"]
    for kw in (dict(keep=w["keep"][0]), dict(keep=w["keep"][:, :0].contiguous()), dict(n_keep=w["n_keep"][:1]), dict(cu_seqlens_q=w["n_keep"]),
               dict(block_table=w["block_table"][:1]), dict(kv_pool=pool.float()), dict(kv_pool=pool[..., :500]), dict(kv_pool=pool[:, :, 0]),
               dict(kv_pool=pool[:, ::2]), dict(kv_pool=pool.cpu()), dict(free_start=i32([0, 0])), dict(seqlens=i32([0])),
               dict(counts=i32([0, 0])), dict(seqlens=w["seqlens_k"]), dict(page_block=0), dict(free_pages=w["block_table"].view(-1)),
               dict(counts=w["free_pages"][:3])):
        with pytest.raises((ValueError, TypeError, smla.SmlaError)):
            smla.sparse_mla_commit_tree(**dict(w, **kw))


# ------------------------------------------------------------------------- speculative steps
def step_state(n_req, heads, page, width, layers, n_pages, cap):
    def ints(*shape, fill=0):
        return torch.full(shape, fill, dtype=torch.int32, device="cuda")
    return dict(lens=ints(n_req), new=ints(n_req), start=ints(1), table=ints(n_req, width, fill=-1),
                free=i32(np.random.default_rng(2).permutation(n_pages)), parents=ints(cap), tokens=ints(cap),
                pool=torch.zeros(layers, n_pages * page, 1, 576, dtype=torch.bfloat16, device="cuda"),
                x=torch.zeros(layers, cap, 576, dtype=torch.bfloat16, device="cuda"),
                q=torch.zeros(layers, cap, heads, 576, dtype=torch.bfloat16, device="cuda"),
                target=torch.ones(cap, 50, device="cuda") / 50, draft=torch.ones(cap, 50, device="cuda") / 50,
                accept_u=torch.zeros(cap, device="cuda"), sample_u=torch.zeros(n_req, device="cuda"))


def step(s, page, words, max_keep, rope):
    """One speculative step: pages, masks, rows and attention of every layer, verification, commit."""
    k, cu, slots, _, counts = smla.sparse_mla_plan_pages(s["lens"], s["new"], s["table"], s["free"], s["parents"].numel(),
                                                         page_block=page, free_start=s["start"])
    mask, pos = smla.sparse_mla_plan_tree(s["parents"], cu, k, words)
    outs = []
    for pool, x, q in zip(s["pool"], s["x"], s["q"]):
        q = q.clone()
        smla.sparse_mla_append_kv(x[:, :512], x[:, 512:], slots, pool, positions=pos, rope=rope, q_pe=q[..., 512:], q=q)
        outs.append((q, *smla.sparse_mla_tree_fwd_paged(q, pool, s["table"], cu, k, mask, page_block=page)))
    keep, out_tokens, n_keep = smla.sparse_mla_verify_tree(s["target"], s["tokens"], s["parents"], cu, s["accept_u"], s["sample_u"],
                                                           max_keep, draft_probs=s["draft"])
    lens, c = smla.sparse_mla_commit_tree(keep, n_keep, cu, k, s["table"], s["pool"], page_block=page, free_pages=s["free"],
                                          free_start=counts[1:2])
    s["lens"].copy_(lens)
    s["start"].copy_(c[1:2])
    return dict(k=k, cu=cu, slots=slots, mask=mask, pos=pos, counts=counts, outs=outs, keep=keep, out_tokens=out_tokens, n_keep=n_keep, c=c)


def fill_step(s, rng, sizes, kind):
    n = int(sum(sizes))
    s["new"].copy_(i32(sizes))
    parents = [p for m in sizes for p in random_parents(rng, m, kind)]
    s["parents"][:n] = i32(parents)
    s["tokens"][:n] = i32(rng.integers(0, 50, n))
    for name in ("x", "q"):
        s[name].copy_(torch.from_numpy(rng.standard_normal(tuple(s[name].shape), dtype=np.float32)))
    for name in ("target", "draft"):
        s[name].copy_(torch.from_numpy(rng.random(tuple(s[name].shape), dtype=np.float32)))
        s[name] /= s[name].sum(-1, keepdim=True)
    for name in ("accept_u", "sample_u"):
        s[name].copy_(torch.from_numpy(rng.random(tuple(s[name].shape), dtype=np.float32)))


def test_speculative_steps_together():
    """Prompts (chains) and trees over several steps.  After each one the cache holds, position by position, the rows of the
    tokens that were kept, as if those alone had been appended; the kept nodes' attention is the causal attention
    over that cache; no page is lost or handed out twice."""
    n_req, heads, page, width, layers, n_pages, cap = 5, 16, 8, 20, 2, 90, 220
    rng, rope = np.random.default_rng(5), rope_table(256)
    s = step_state(n_req, heads, page, width, layers, n_pages, cap)
    plain = torch.zeros_like(s["pool"])            # the same table, rows appended one by one
    history = [[] for _ in range(n_req)]
    for sizes, kind, words in (([40, 3, 17, 60, 8], "chain", 2), ([8, 16, 1, 40, 0], "tree", 2), ([7] * n_req, "star", 1),
                               ([33, 5, 12, 9, 24], "tree", 2), ([9] * n_req, "comb", 1)):
        fill_step(s, rng, sizes, kind)
        if kind == "chain":
            s["accept_u"].zero_()                  # a prompt is kept whole
            s["target"].copy_(torch.nn.functional.one_hot(s["tokens"].roll(-1).long(), 50).float())
            s["draft"].copy_(s["target"])
        old = s["lens"].tolist()
        got = step(s, page, words, 64, rope)
        cu, table = got["cu"].tolist(), s["table"]
        for b, m in enumerate(sizes):
            n_keep = int(got["n_keep"][b])
            path = got["keep"][b, :n_keep].tolist()
            assert (n_keep >= 1) == (m > 0) and (kind != "chain" or n_keep == m)
            for i, node in enumerate(path):
                history[b].append((s["x"][:, cu[b] + node].clone(), old[b] + i))
                assert int(got["pos"][cu[b] + node]) == old[b] + i
            assert int(s["lens"][b]) == len(history[b])
            if not history[b]:
                continue
            xs = torch.stack([x for x, _ in history[b]], 1)                       # [layers, length, 576]
            pos = i32([at for _, at in history[b]])
            rows = table[b, pos.long() // page].long() * page + pos.long() % page
            for layer in range(layers):
                smla.sparse_mla_append_kv(xs[layer, :, :512], xs[layer, :, 512:], rows.to(torch.int32), plain[layer], positions=pos, rope=rope)
                assert torch.equal(s["pool"][layer, rows], plain[layer, rows])
                if n_keep:
                    q, out, lse, top = (t[cu[b]:cu[b + 1]][path].contiguous() for t in got["outs"][layer])
                    o2, l2, t2 = smla.sparse_mla_chunk_fwd_paged(q, s["pool"][layer], table[b:b + 1].contiguous(), i32([0, n_keep]),
                                                                 s["lens"][b:b + 1].clone(), page_block=page)
                    # each side is within its roundings of the same values: weights and output rounded to bf16
                    v = float(s["pool"][layer, rows].float().abs().max())
                    assert float((out.float() - o2.float()).abs().max()) <= 2 * 2.1 * U16 * v
                    assert float((lse - l2).abs().max()) <= 1e-3 and float((top - t2).abs().max()) <= 1e-3
        assert int(got["counts"][2]) == 0 and int(got["c"][2]) == 0
        held = [p for b in range(n_req) for p in table[b, :-(-int(s["lens"][b]) // page)].tolist()]
        assert sorted(held + s["free"][int(s["start"]):].tolist()) == list(range(n_pages))


def test_speculative_step_in_one_graph():
    """A whole step captured once and replayed over steps whose trees, lengths and inputs change in place, against the
    same steps run call by call."""
    n_req, heads, page, width, layers, n_pages, cap = 4, 16, 8, 20, 2, 80, 90
    rope = rope_table(256)
    a, b = (step_state(n_req, heads, page, width, layers, n_pages, cap) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(b, page, 2, 9, rope)
    b2 = step_state(n_req, heads, page, width, layers, n_pages, cap)
    for key in b:
        b[key].copy_(b2[key])
    for i, (sizes, kind) in enumerate((([20, 3, 33, 1], "chain"), ([8, 16, 1, 30], "tree"), ([5, 0, 9, 7], "star"), ([0] * 4, "tree"))):
        for s in (a, b):
            fill_step(s, np.random.default_rng(i), sizes, kind)
        want = step(a, page, 2, 9, rope)
        graph.replay()
        n = sum(sizes)
        for name in ("k", "cu", "slots", "pos", "mask", "counts", "keep", "out_tokens", "n_keep", "c"):
            assert torch.equal(want[name], captured[name]), name
        for u, v in zip(want["outs"], captured["outs"]):
            assert all(torch.equal(x[:n], y[:n]) for x, y in zip(u, v))
        assert all(torch.equal(a[key], b[key]) for key in ("lens", "start", "table", "free", "pool"))


FIRST_CALLS_CAPTURED = """
import sys
sys.path.insert(0, sys.argv[1])
import torch, sparse_mla_attention_fwd_gb300 as smla
torch.manual_seed(0)
def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")
pool, q = torch.randn(4 * 64, 1, 576, device="cuda").to(torch.bfloat16), torch.randn(5, 16, 576, device="cuda").to(torch.bfloat16)
parents, cu, lens, table, tokens = ints([-1, 0, 0, -1, 0]), ints([0, 3, 5]), ints([103, 66]), ints([[0, 1], [2, 3]]), ints([1, 2, 3, 4, 5])
probs, u = torch.rand(5, 77, device="cuda"), torch.rand(5, device="cuda")
torch.cuda.synchronize()
def step():
    mask, pos = smla.sparse_mla_plan_tree(parents, cu, lens, 1)
    out = smla.sparse_mla_tree_fwd_paged(q, pool, table, cu, lens, mask)
    kept = smla.sparse_mla_verify_tree(probs, tokens, parents, cu, u, u[:2], 3, draft_probs=probs)
    return [mask, pos, *out, *kept, *smla.sparse_mla_commit_tree(kept[0], kept[2], cu, lens, table, None)]
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
