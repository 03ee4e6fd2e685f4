"""Cases for the paged-cache operators: placing a step's new tokens in the cache's pages, appending
their latent rows, and dense attention of the new tokens over the paged cache.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits) or, with
``own`` set, through the framework's entry points.  ``exact`` computes the floating outputs in 64
bits, request by request, from the definitions.
"""
import random

import torch

own = False

D_V = 512        # value width of a latent row
D_ROPE = 64      # rotary columns behind it when d_qk is 576
EPS = 1e-6


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a small server: eight requests, one token each
        dict(name="plan, 8 requests decode", op="plan", n_req=8, old_max=4096, new_max=1, page=64, max_blocks=64,
             pad=0),
        # a decode step of the benchmark's batch, padded to a captured graph's 300 tokens
        dict(name="plan, 256 requests padded", op="plan", n_req=256, old_max=4000, new_max=1, page=64, max_blocks=64,
             pad=44),
        # a mixed step: ragged prefill chunks next to decode tokens, small pages
        dict(name="plan, 700 ragged chunks", op="plan", n_req=700, old_max=9000, new_max=150, page=16, max_blocks=600,
             pad=100),
        # decode: the queries' rotary part of all 128 heads and one new row per request
        dict(name="append, 256 tokens, 128 heads", op="append", n=256, d_qk=576, heads=128, pool_rows=16384, pad=0),
        # a prefill chunk of 8192 tokens on one of eight tensor-parallel ranks
        dict(name="append, 8192 tokens, 16 heads", op="append", n=8192, d_qk=576, heads=16, pool_rows=16384, pad=77),
        # a cache without rotary columns; an odd number of tokens
        dict(name="append, 1021 tokens, no rope", op="append", n=1021, d_qk=512, heads=0, pool_rows=8192, pad=5),
        # one user decoding: latency
        dict(name="attention, 1 token", op="attention", n_req=1, q_min=1, q_max=1, kv_min=1500, kv_max=1500, heads=128,
             d_qk=576, page=64, causal=True, sink=False),
        # the benchmark's decode batch with dense attention, ragged lengths
        dict(name="attention, 256 requests decode", op="attention", n_req=256, q_min=1, q_max=1, kv_min=1024,
             kv_max=4096, heads=128, d_qk=576, page=64, causal=True, sink=False),
        # long contexts on one of eight tensor-parallel ranks, two speculative tokens at most
        dict(name="attention, long, 16 heads", op="attention", n_req=48, q_min=1, q_max=2, kv_min=9000, kv_max=32768,
             heads=16, d_qk=576, page=64, causal=True, sink=True),
        # chunked prefill behind cached prefixes
        dict(name="attention, 4 chunks of 512", op="attention", n_req=4, q_min=300, q_max=512, kv_min=2048, kv_max=8192,
             heads=64, d_qk=576, page=64, causal=True, sink=False),
        # the last chunk of a long prompt, all heads
        dict(name="attention, chunk of 2048", op="attention", n_req=1, q_min=2048, q_max=2048, kv_min=8192, kv_max=8192,
             heads=128, d_qk=576, page=64, causal=True, sink=False),
        # odd sizes: 20 heads, no rotary columns, small pages, every cached key visible
        dict(name="attention, odd, not causal", op="attention", n_req=5, q_min=7, q_max=133, kv_min=150, kv_max=1999,
             heads=20, d_qk=512, page=16, causal=False, sink=True),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["plan", "append", "attention", "attention"])
    if kind == "plan":
        old, new, page = _between(rng, 100, 9000), _between(rng, 1, 150), rng.choice([16, 32, 64, 100])
        return dict(op="plan", n_req=_between(rng, 8, 700), old_max=old, new_max=new, page=page,
                    max_blocks=-(-(old + new) // page) + rng.randint(0, 8), pad=rng.randint(0, 100))
    if kind == "append":
        d_qk, n = rng.choice([512, 576, 576]), _between(rng, 200, 8192)
        heads = 0 if d_qk == 512 else rng.choice([8, 16, 32, 64, 128])
        if heads:
            n = min(n, max(200, 8192 * 16 // heads))
        return dict(op="append", n=n, d_qk=d_qk, heads=heads, pool_rows=64 * rng.randint(130, 256), pad=rng.randint(0, 90))
    heads, d_qk, page = rng.choice([8, 16, 20, 32, 64, 96, 128]), rng.choice([512, 576, 576]), rng.choice([16, 32, 64, 100])
    kv_max = _between(rng, 400, 32768)
    kv_min = max(150, int(kv_max * rng.uniform(0.2, 1.0)))
    if rng.random() < 0.5:
        q_max = rng.randint(1, 4)
        n_req = min(_between(rng, 1, 256), max(1, 1000000 // kv_max))
        q_min = 1
    else:
        q_max = _between(rng, 16, 2048)
        n_req = _between(rng, 1, 8)
        q_min = max(1, int(q_max * rng.uniform(0.3, 1.0)))
    q_max = min(q_max, kv_min)
    # the padded scores of the plain form, and the products
    while n_req * q_max * heads * kv_max > 2.0e9:
        if n_req > 1:
            n_req -= 1
        else:
            q_max = max(1, q_max // 2)
    return dict(op="attention", n_req=n_req, q_min=min(q_min, q_max), q_max=q_max, kv_min=kv_min, kv_max=kv_max, heads=heads,
                d_qk=d_qk, page=page, causal=rng.random() < 0.8, sink=rng.random() < 0.3)


def _lengths(case):
    """The requests' lengths: a property of the case, whatever the seed of its values."""
    rng = random.Random("%(op)s %(n_req)d %(page)d" % case)
    if case["op"] == "plan":
        new = [1 if case["new_max"] == 1 or rng.random() < 0.3 else rng.randint(0, case["new_max"]) for _ in range(case["n_req"])]
        return [rng.randint(0, case["old_max"]) for _ in new], new
    q = [rng.randint(case["q_min"], case["q_max"]) for _ in range(case["n_req"])]
    k = [rng.randint(case["kv_min"], case["kv_max"]) for _ in q]
    q[0], k[-1] = case["q_max"], case["kv_max"]
    return q, k


# ------------------------------------------------------------------------------------ inputs
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    s = dict(case)
    if case["op"] == "plan":
        old, new = _lengths(case)
        page = case["page"]
        held = [-(-n // page) for n in old]
        n_free = sum(-(-(n + m) // page) for n, m in zip(old, new)) - sum(held) + 32
        pages = torch.randperm(sum(held) + n_free, generator=g, device="cuda").to(torch.int32)
        table = torch.full((case["n_req"], case["max_blocks"]), -1, dtype=torch.int32, device="cuda")
        cols = torch.arange(case["max_blocks"], device="cuda")
        table[cols[None, :] < torch.tensor(held, device="cuda")[:, None]] = pages[:sum(held)]
        s.update(seqlens=_ints(old), new_lens=_ints(new), block_table=table, free_pages=pages[sum(held):].contiguous(),
                 n_tokens=sum(new) + case["pad"], free_start=torch.full((1,), 7, dtype=torch.int32, device="cuda"))
        return s
    if case["op"] == "append":
        n, d_qk, heads, rows = case["n"], case["d_qk"], case["heads"], case["pool_rows"]
        x = normal(n, d_qk, scale=2.0)                    # the layer's down projection: latent | rotary key
        buf = normal(rows + 1, 1, d_qk)                   # the plain form puts padding in the row behind the pool
        slots = torch.randperm(rows, generator=g, device="cuda")[:n].to(torch.int32)
        slots[n - case["pad"]:] = -1                      # a padded batch
        s.update(c_kv=x[:, :D_V], k_pe=None, slots=slots, rows_and_spare=buf, kv_pool=buf[:rows],
                 norm_weight=(1.0 + 0.1 * torch.randn(D_V, generator=g, device="cuda")).to(torch.bfloat16),
                 positions=None, rope=None, q_pe=None, q=None)
        if d_qk > D_V:
            max_pos = 16384
            inv = 10000.0 ** (-torch.arange(D_ROPE // 2, device="cuda", dtype=torch.float64) * 2 / D_ROPE)
            angle = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * inv
            positions = torch.randint(0, max_pos, (n,), generator=g, device="cuda").to(torch.int32)
            positions[n - case["pad"]:] = -1
            up = normal(n, heads, 128 + D_ROPE)           # the queries' up projection: without | with position
            s.update(k_pe=x[:, D_V:], positions=positions, rope=torch.cat([angle.cos(), angle.sin()], 1).float(),
                     q_pe=up[..., 128:], q=normal(n, heads, d_qk))
        return s
    q_lens, k_lens = _lengths(case)
    page, d_qk, heads = case["page"], case["d_qk"], case["heads"]
    held = [-(-n // page) for n in k_lens]
    n_pages = sum(held) + 3
    table = torch.full((case["n_req"], max(held) + 1), -1, dtype=torch.int32, device="cuda")
    cols = torch.arange(max(held) + 1, device="cuda")
    table[cols[None, :] < torch.tensor(held, device="cuda")[:, None]] = \
        torch.randperm(n_pages, generator=g, device="cuda")[:sum(held)].to(torch.int32)
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    s.update(q=normal(cu[-1], heads, d_qk), kv_pool=normal(n_pages * page, 1, d_qk), block_table=table,
             cu_seqlens_q=_ints(cu), seqlens_k=_ints(k_lens), max_q=max(q_lens), max_k=max(k_lens),
             attn_sink=torch.randn(heads, generator=g, device="cuda") if case["sink"] else None)
    return s


# ------------------------------------------------------------------------------- plain forms
def _plan_plain(s):
    page, table, width = s["page"], s["block_table"], s["block_table"].shape[1]
    old, new = s["seqlens"].clamp(min=0).long(), s["new_lens"].clamp(min=0).long()
    end = new.cumsum(0).clamp(max=s["n_tokens"])
    cu = torch.cat([end.new_zeros(1), end])
    length = old + cu[1:] - cu[:-1]
    first = ((old + page - 1) // page).clamp(max=width)
    last = ((length + page - 1) // page).clamp(max=width)
    before = (last - first).cumsum(0) - (last - first)
    col = torch.arange(width, device="cuda")[None, :]
    at = s["free_start"].long() + before[:, None] + col - first[:, None]
    n_free = s["free_pages"].shape[0]
    page_of = torch.where(at < n_free, s["free_pages"][at.clamp(0, n_free - 1)], -1)
    table.copy_(torch.where((col >= first[:, None]) & (col < last[:, None]), page_of, table))
    t = torch.arange(s["n_tokens"], device="cuda")
    real = t < cu[-1]
    req = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=old.shape[0] - 1)
    pos = torch.where(real, old[req] + t - cu[req], -1)
    entry = table[req, (pos // page).clamp(0, width - 1)]
    slots = torch.where(real & (pos < width * page) & (entry >= 0), entry * page + pos % page, -1)
    need = (last - first).sum()
    room = (n_free - s["free_start"].long()[0]).clamp(min=0)
    taken = torch.minimum(need, room)
    counts = torch.stack([cu[-1], s["free_start"].long()[0] + taken, need - taken])
    return dict(seqlens_k=length.int(), cu_seqlens_q=cu.int(), slots=slots.int(), positions=pos.int(), counts=counts.int(),
                block_table=table)


def _rotate_plain(x, cos, sin):
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).reshape(x.shape)


def _append_plain(s):
    c = s["c_kv"].float()
    row = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["norm_weight"].float()
    real = s["slots"] >= 0
    if s["rope"] is not None:
        real = real & (s["positions"] >= 0)
        cos, sin = s["rope"][s["positions"].clamp(min=0).long()].split(D_ROPE // 2, -1)
        row = torch.cat([row, _rotate_plain(s["k_pe"].float(), cos, sin)], -1)
        turned = _rotate_plain(s["q_pe"].float(), cos[:, None], sin[:, None]).to(torch.bfloat16)
        tail = s["q"][..., D_V:]
        tail.copy_(torch.where((s["positions"] >= 0)[:, None, None], turned, tail))
    buf = s["rows_and_spare"]
    buf[torch.where(real, s["slots"].long(), buf.shape[0] - 1), 0] = row.to(torch.bfloat16)
    return [s["kv_pool"]] + ([] if s["q"] is None else [s["q"]])


def _attention_plain(s):
    q, table, cu, page = s["q"], s["block_table"], s["cu_seqlens_q"].long(), s["page"]
    heads, n_req, scale = q.shape[1], table.shape[0], q.shape[2] ** -0.5
    i, j = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_k"], device="cuda")
    q_lens, k_lens = cu[1:] - cu[:-1], s["seqlens_k"].long()
    rows = table[:, j // page].long() * page + j % page
    seen = j < k_lens[:, None]
    kv = torch.where(seen[..., None], s["kv_pool"][:, 0][rows.clamp(min=0)].float(), 0.0)       # [n_req, max_k, d_qk]
    qp = q[(cu[:-1, None] + i).clamp(max=q.shape[0] - 1)].float().reshape(n_req, -1, q.shape[2])  # [n_req, max_q heads, d_qk]
    logits = (qp @ kv.transpose(1, 2)).mul_(scale).reshape(n_req, s["max_q"], heads, -1)
    ok = seen[:, None, :]
    if s["causal"]:
        ok = ok & (j <= (k_lens - q_lens)[:, None, None] + i[:, None])
    logits.masked_fill_(~ok[:, :, None, :], float("-inf"))
    top = logits.amax(-1)
    p = logits.sub_(torch.where(top.isinf(), 0.0, top)[..., None]).exp_()
    total = p.sum(-1)
    den = total if s["attn_sink"] is None else total + (s["attn_sink"] - top).exp()
    o = (p.reshape(n_req, -1, p.shape[-1]) @ kv[..., :D_V]).reshape(n_req, s["max_q"], heads, D_V)
    o = torch.where(total[..., None] > 0, o / den[..., None], 0.0)
    lse = torch.where(total > 0, top + total.log(), float("inf"))
    t = torch.arange(q.shape[0], device="cuda")
    req = torch.searchsorted(cu, t, right=True) - 1
    at = (req, t - cu[req])
    return o[at].to(torch.bfloat16), lse[at], top[at]


def run(s):
    if own:
        import sparse_mla_attention_fwd_gb300 as smla
        if s["op"] == "plan":
            names = ("seqlens_k", "cu_seqlens_q", "slots", "positions", "counts")
            got = smla.sparse_mla_plan_pages(s["seqlens"], s["new_lens"], s["block_table"], s["free_pages"], s["n_tokens"],
                                             page_block=s["page"], free_start=s["free_start"])
            return dict(zip(names, got), block_table=s["block_table"])
        if s["op"] == "append":
            smla.sparse_mla_append_kv(s["c_kv"], s["k_pe"], s["slots"], s["kv_pool"], norm_weight=s["norm_weight"], eps=EPS,
                                      positions=s["positions"], rope=s["rope"], q_pe=s["q_pe"], q=s["q"])
            return [s["kv_pool"]] + ([] if s["q"] is None else [s["q"]])
        return smla.sparse_mla_chunk_fwd_paged(s["q"], s["kv_pool"], s["block_table"], s["cu_seqlens_q"], s["seqlens_k"],
                                               page_block=s["page"], causal=s["causal"], attn_sink=s["attn_sink"])
    return {"plan": _plan_plain, "append": _append_plain, "attention": _attention_plain}[s["op"]](s)


# ------------------------------------------------------------------------- what has to be done
def _visible(case):
    q_lens, k_lens = _lengths(case)
    if not case["causal"]:
        return sum(n * m for n, m in zip(q_lens, k_lens))
    return sum(n * m - n * (n - 1) // 2 for n, m in zip(q_lens, k_lens))


def work(case):
    if case["op"] == "plan":
        old, new = _lengths(case)
        pages = sum(-(-(n + m) // case["page"]) + -(-n // case["page"]) * -1 for n, m in zip(old, new))
        part = sum(1 for n, m in zip(old, new) if m and n % case["page"])
        return dict(bytes=case["n_req"] * 16 + (sum(new) + case["pad"]) * 8 + pages * 8 + part * 4 + 20, flops=0)
    if case["op"] == "append":
        n, real, d = case["n"], case["n"] - case["pad"], case["d_qk"]
        size = real * d * 2 * 2 + n * 4 + D_V * 2
        flops = real * D_V * 4
        if d > D_V:
            size += n * 4 + real * (D_ROPE * 4 + case["heads"] * D_ROPE * 2 * 2)
            flops += real * (case["heads"] + 1) * D_ROPE * 3
        return dict(bytes=size, flops=flops)
    q_lens, k_lens = _lengths(case)
    n, d = sum(q_lens), case["d_qk"]
    rows = n * case["heads"]
    return dict(bytes=sum(k_lens) * d * 2 + rows * (d + D_V) * 2 + rows * 8 + sum(-(-k // case["page"]) for k in k_lens) * 4,
                flops=_visible(case) * case["heads"] * 2 * (d + D_V))


# ---------------------------------------------------------------------------------- in 64 bits
def _exact_append(s):
    """Row by row of the definition: y_d = c_d w_d / sqrt(mean c^2 + eps); each pair (x, y) as the
    complex number x + iy times exp(i angle)."""
    pool, slots = s["kv_pool"].double(), s["slots"].long()
    keep = slots >= 0
    c = s["c_kv"].double()[keep]
    new = c * s["norm_weight"].double() / ((c ** 2).sum(1, keepdim=True) / D_V + EPS).sqrt()
    q = None
    if s["rope"] is not None:
        turn = s["rope"].double()[s["positions"].long()[keep]]
        turn = torch.complex(turn[:, :D_ROPE // 2], turn[:, D_ROPE // 2:])

        def rotated(x):
            z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], -1, 2).contiguous())
            return torch.view_as_real(z * turn.reshape(turn.shape[0], *([1] * (x.dim() - 2)), -1)).flatten(-2)

        new = torch.cat([new, rotated(s["k_pe"][keep])], 1)
        q = s["q"].double()
        q[keep, :, D_V:] = rotated(s["q_pe"][keep])
    pool[slots[keep], 0] = new
    return [pool] + ([] if q is None else [q])


def _exact_attention(s):
    q, cu = s["q"], s["cu_seqlens_q"].tolist()
    out = torch.zeros(q.shape[0], q.shape[1], D_V, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], float("inf"), dtype=torch.float64, device="cuda")
    top = torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
    for b, n_k in enumerate(s["seqlens_k"].tolist()):
        pages = s["block_table"][b, :-(-n_k // s["page"])].long()
        kv = s["kv_pool"].reshape(-1, s["page"], q.shape[2])[pages].reshape(-1, q.shape[2])[:n_k].double()
        for t0 in range(cu[b], cu[b + 1], 64):
            t1 = min(t0 + 64, cu[b + 1])
            z = torch.einsum("thd,kd->thk", q[t0:t1].double(), kv) / q.shape[2] ** 0.5
            if s["causal"]:
                last = torch.arange(t0, t1, device="cuda") - cu[b + 1] + n_k         # the token's own position
                z[(torch.arange(n_k, device="cuda") > last[:, None])[:, None].expand_as(z)] = float("-inf")
            top[t0:t1] = z.max(-1).values
            lse[t0:t1] = torch.logsumexp(z, -1)
            full = lse[t0:t1] if s["attn_sink"] is None else torch.logaddexp(lse[t0:t1], s["attn_sink"].double()[None, :])
            out[t0:t1] = torch.einsum("thk,kd->thd", (z - full[..., None]).exp(), kv[:, :D_V])
    return out, lse, top


def exact(case, seed):
    if case["op"] == "plan" or (case["op"] == "attention" and work(case)["flops"] > 8e12):
        return None
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)
