"""Cases for the operators of a speculative step on the paged cache: planning a tree of drafted tokens,
attention of the tree over the cache, verification against the target's probabilities, and committing the
accepted tokens (rows moved together, pages given back).

``run`` computes an operator in its plain form (elementary torch operations) or, with ``own`` set, through the
framework's entry points.  ``exact`` computes the attention in 64 bits, request by request, from the definition;
the other operators give whole numbers and copied rows.
"""
import random

import torch

own = False

D_V = 512        # value width of a latent row


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a small server: eight requests, trees of up to eight nodes
        dict(name="plan, 8 trees of 8", op="plan", n_req=8, n_min=5, n_max=8, old_max=4000, pad=0),
        # a large batch of wide trees, padded to a captured graph's size
        dict(name="plan, 300 trees of 64", op="plan", n_req=300, n_min=33, n_max=64, old_max=9000, pad=77),
        # one user: latency
        dict(name="attention, 1 tree of 8", op="attention", n_req=1, n_min=8, n_max=8, kv_min=1500, kv_max=1500,
             heads=128, d_qk=576, page=64, sink=False),
        # a decode batch, all heads on one GPU
        dict(name="attention, 64 trees", op="attention", n_req=64, n_min=6, n_max=16, kv_min=1024, kv_max=4096,
             heads=128, d_qk=576, page=64, sink=False),
        # long contexts on one of eight tensor-parallel ranks
        dict(name="attention, long, 16 heads", op="attention", n_req=24, n_min=3, n_max=8, kv_min=9000, kv_max=32768,
             heads=16, d_qk=576, page=64, sink=True),
        # odd sizes: 20 heads, no rotary columns, small pages, trees of more than one mask word
        dict(name="attention, odd, wide trees", op="attention", n_req=5, n_min=17, n_max=61, kv_min=150, kv_max=1999,
             heads=20, d_qk=512, page=16, sink=True),
        # one user, a chain of drafts with the draft model's probabilities: latency
        dict(name="verify, 1 chain of 5", op="verify", n_req=1, n_min=5, n_max=5, vocab=32000, siblings=1, probs=True),
        # a large batch of chains, large vocabulary
        dict(name="verify, 256 chains of 6", op="verify", n_req=256, n_min=3, n_max=6, vocab=128000, siblings=1,
             probs=True),
        # trees of the likeliest tokens (no draft probabilities), odd vocabulary
        dict(name="verify, 48 trees of 24", op="verify", n_req=48, n_min=11, n_max=24, vocab=50001, siblings=4,
             probs=False),
        # trees of tokens drawn from the draft model: several rejections at a node
        dict(name="verify, 32 drawn trees of 16", op="verify", n_req=32, n_min=9, n_max=16, vocab=100003, siblings=4,
             probs=True),
        # a small server, one layer's cache
        dict(name="commit, 8 trees, 1 layer", op="commit", n_req=8, n_min=5, n_max=8, old_max=300, page=64, layers=1,
             d_qk=576),
        # a large batch, the caches of all layers at once
        dict(name="commit, 120 trees, 24 layers", op="commit", n_req=120, n_min=9, n_max=32, old_max=300, page=64,
             layers=24, d_qk=576),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["plan", "attention", "attention", "verify", "commit"])
    if kind == "plan":
        n_max = _between(rng, 2, 128)
        return dict(op="plan", n_req=min(_between(rng, 4, 400), 19200 // n_max), n_min=max(1, int(n_max * rng.uniform(0.2, 1.0))),
                    n_max=n_max, old_max=_between(rng, 100, 9000), pad=rng.randint(0, 100))
    if kind == "verify":
        probs, siblings = rng.random() < 0.6, rng.choice([1, 2, 4])
        n_max = rng.randint(2, 24)
        vocab = _between(rng, 1000, 150000)
        n_req = _between(rng, 1, 256)
        # the plain form passes over a row of every request for each node
        while n_req * n_max * vocab > 190000000:
            n_req = max(1, n_req * 2 // 3)
        return dict(op="verify", n_req=n_req, n_min=max(1, int(n_max * rng.uniform(0.3, 1.0))), n_max=n_max, vocab=vocab,
                    siblings=siblings, probs=probs)
    if kind == "commit":
        n_max, layers = rng.randint(2, 64), _between(rng, 1, 24)
        n_req = min(_between(rng, 4, 256), max(4, 2880 // layers))
        return dict(op="commit", n_req=n_req, n_min=max(1, int(n_max * rng.uniform(0.3, 1.0))), n_max=n_max,
                    old_max=_between(rng, 30, 300), page=rng.choice([16, 32, 64, 100]), layers=layers,
                    d_qk=rng.choice([512, 576, 576]))
    heads, d_qk, page = rng.choice([8, 16, 20, 32, 64, 96, 128]), rng.choice([512, 576, 576]), rng.choice([16, 32, 64, 100])
    n_max, kv_max = _between(rng, 2, 70), _between(rng, 400, 32768)
    n_req = min(_between(rng, 1, 128), max(1, 800000 // kv_max))
    # the padded scores of the plain form, and the products
    while n_req * n_max * heads * kv_max > 5.0e8:
        if n_req > 1:
            n_req -= 1
        else:
            n_max = max(2, n_max // 2)
            kv_max = max(400, kv_max * 3 // 4)
    return dict(op="attention", n_req=n_req, n_min=max(1, int(n_max * rng.uniform(0.3, 1.0))), n_max=n_max,
                kv_min=max(n_max, int(kv_max * rng.uniform(0.2, 1.0))), kv_max=kv_max, heads=heads, d_qk=d_qk, page=page,
                sink=rng.random() < 0.3)


def _sizes(case):
    """Nodes and keys (the new tokens' own among them) of each request: a property of the case, whatever the seed."""
    rng = random.Random("%(op)s %(n_req)d %(n_max)d" % case)
    n = [rng.randint(case["n_min"], case["n_max"]) for _ in range(case["n_req"])]
    n[0] = case["n_max"]
    if case["op"] == "attention":
        k = [rng.randint(case["kv_min"], case["kv_max"]) for _ in n]
        k[-1] = case["kv_max"]
    else:
        k = [rng.randint(0, case.get("old_max", 0)) + m for m in n]
    return n, k


def _trees(case, seed):
    """Parents of each request's nodes (index within the request, -1 for the root, node 0), and each node's
    place among its siblings."""
    rng = random.Random("tree %(op)s %(n_req)d %(n_max)d" % case + " %d" % seed)
    most = case.get("siblings", 4)
    parents, places = [], []
    for m in _sizes(case)[0]:
        par, place, children = [-1], [0], [0] * m
        for i in range(1, m):
            free = [j for j in range(max(0, i - 8), i) if children[j] < most]
            j = free[-1] if most == 1 or rng.random() < 0.4 else rng.choice(free)
            par.append(j)
            place.append(children[j])
            children[j] += 1
        parents.append(par)
        places.append(place)
    return parents, places


def _flat(lists):
    return [x for one in lists for x in one]


def _sums(values):
    out = [0]
    for v in values:
        out.append(out[-1] + v)
    return out


# ------------------------------------------------------------------------------------ inputs
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(held, n_pages, width, page_ids):
    table = torch.full((len(held), width), -1, dtype=torch.int32, device="cuda")
    cols = torch.arange(width, device="cuda")
    table[cols[None, :] < torch.tensor(held, device="cuda")[:, None]] = page_ids[:sum(held)]
    return table


def _pack(seen):
    """Rows of truth values as 32-bit words, lowest bit first."""
    bits = seen.unflatten(-1, (-1, 32)).long() << torch.arange(32, device="cuda")
    return bits.sum(-1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s, (n, k) = dict(case), _sizes(case)
    parents, places = _trees(case, seed)
    cu, words = _sums(n), -(-case["n_max"] // 32)
    s.update(cu_seqlens_q=_ints(cu), n_tok=cu[-1], max_n=max(n), words=words)
    if case["op"] == "plan":
        old = torch.randint(0, case["old_max"] + 1, (len(n),), generator=g, device="cuda").to(torch.int32)
        s.update(parents=_ints(_flat(parents) + [0] * case["pad"]), seqlens_k=old + _ints(n))
        return s
    if case["op"] == "attention":
        page, held = case["page"], [-(-m // case["page"]) for m in k]
        n_pages = sum(held) + 3
        table = _table(held, n_pages, max(held) + 1, torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32))
        seen = torch.zeros(len(n), max(n), words * 32, dtype=torch.bool)
        for b, par in enumerate(parents):
            for i, j in enumerate(par):
                if j >= 0:
                    seen[b, i] = seen[b, j]
                seen[b, i, i] = True
        rows = torch.tensor([b * max(n) + i for b, m in enumerate(n) for i in range(m)], device="cuda")
        s.update(q=normal(cu[-1], case["heads"], case["d_qk"]).to(torch.bfloat16),
                 kv_pool=normal(n_pages * page, 1, case["d_qk"]).to(torch.bfloat16), block_table=table, seqlens_k=_ints(k),
                 max_k=max(k), tree_mask=_pack(seen.cuda()).flatten(0, 1)[rows].contiguous(),
                 attn_sink=normal(case["heads"]) if case["sink"] else None)
        return s
    if case["op"] == "verify":
        vocab, most = case["vocab"], case["siblings"]
        logits = normal(cu[-1], vocab) * 4.0
        near = logits + normal(cu[-1], vocab) * 1.3            # the draft model's
        target = logits.softmax(-1)
        flat, place = _flat(parents), torch.tensor(_flat(places), device="cuda")
        of = torch.tensor([cu[b] + max(j, 0) for b, par in enumerate(parents) for j in par], device="cuda")
        draft = near.softmax(-1) if case["probs"] else None
        chosen = torch.multinomial(draft, most, replacement=True, generator=g) if case["probs"] else near.topk(most, -1).indices
        s.update(target_probs=target, draft_probs=draft, tokens=chosen[of, place].to(torch.int32), parents=_ints(flat),
                 accept_u=torch.rand(cu[-1], generator=g, device="cuda"), sample_u=torch.rand(len(n), generator=g, device="cuda"),
                 max_keep=max(n))
        return s
    rng, page, width = random.Random("keep %d" % seed), case["page"], -(-(case["old_max"] + case["n_max"]) // case["page"]) + 1
    held = [-(-m // page) for m in k]
    n_pages, most = sum(held) + 5, min(case["n_max"], 9)
    page_ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    keep, n_keep = [], []
    for m in n:
        path = [0] + sorted(rng.sample(range(1, m), rng.randint(0, min(m, most) - 1)))
        n_keep.append(-1 if rng.random() < 0.05 else len(path))           # -1: the request is done
        keep.append(path + [-1] * (most - len(path)))
    s.update(keep=_ints(keep), n_keep=_ints(n_keep), seqlens_k=_ints(k), block_table=_table(held, n_pages, width, page_ids),
             kv_pool=torch.cat([normal(1, n_pages * page, 1, case["d_qk"]).to(torch.bfloat16) for _ in range(case["layers"])]),
             free_pages=page_ids.clone(), free_start=_ints([sum(held)]))
    return s


# ------------------------------------------------------------------------------- plain forms
def _padded(s, x, fill):
    """[n_tok] -> [n_req, max_n]."""
    cu = s["cu_seqlens_q"].long()
    i = torch.arange(s["max_n"], device="cuda")
    return torch.where(i < (cu[1:] - cu[:-1])[:, None], x[(cu[:-1, None] + i).clamp(max=x.shape[0] - 1)], fill)


def _plan_plain(s):
    n, words, cu = s["max_n"], s["words"], s["cu_seqlens_q"].long()
    up = _padded(s, s["parents"], -1)
    i = torch.arange(n, device="cuda")
    step = (up[..., None] == i).double() + torch.eye(n, device="cuda", dtype=torch.float64)
    seen = torch.linalg.matrix_power(step, n) > 0                       # who is reached in up to n steps
    wide = torch.zeros(*seen.shape[:2], words * 32, dtype=torch.bool, device="cuda")
    wide[..., :n] = seen
    n_q = cu[1:] - cu[:-1]
    at = (s["seqlens_k"] - n_q)[:, None] + seen.sum(-1) - 1
    t = torch.arange(s["parents"].shape[0], device="cuda")
    real = t < cu[-1]
    req = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=n_q.shape[0] - 1)
    own_row = (req, (t - cu[req]).clamp(max=n - 1))
    return dict(tree_mask=torch.where(real[:, None], _pack(wide)[own_row], 0), positions=torch.where(real, at[own_row], -1).int())


def _attention_plain(s):
    q, table, cu, page = s["q"], s["block_table"], s["cu_seqlens_q"].long(), s["page"]
    heads, n_req, scale = q.shape[1], table.shape[0], q.shape[2] ** -0.5
    i, j = torch.arange(s["max_n"], device="cuda"), torch.arange(s["max_k"], device="cuda")
    n_q, n_k = cu[1:] - cu[:-1], s["seqlens_k"].long()
    rows = table[:, j // page].long() * page + j % page
    seen = j < n_k[:, None]
    kv = torch.where(seen[..., None], s["kv_pool"][:, 0][rows.clamp(min=0)].float(), 0.0)         # [n_req, max_k, d_qk]
    at = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    logits = (q[at].float().reshape(n_req, -1, q.shape[2]) @ kv.transpose(1, 2)).mul_(scale).reshape(n_req, s["max_n"], heads, -1)
    new = j - (n_k - n_q)[:, None]                                                                # which new token a key is
    word = s["tree_mask"][at].gather(2, (new.clamp(0, s["words"] * 32 - 1) // 32)[:, None].expand(-1, s["max_n"], -1))
    ok = seen[:, None] & ((new < 0)[:, None] | ((word >> (new.clamp(min=0) % 32)[:, None]) & 1 > 0))
    logits.masked_fill_(~ok[:, :, None, :], float("-inf"))
    top = logits.amax(-1)
    p = logits.sub_(torch.where(top.isinf(), 0.0, top)[..., None]).exp_()
    total = p.sum(-1)
    den = total if s["attn_sink"] is None else total + (s["attn_sink"] - top).exp()
    o = (p.reshape(n_req, -1, p.shape[-1]) @ kv[..., :D_V]).reshape(n_req, s["max_n"], heads, D_V)
    o = torch.where(total[..., None] > 0, o / den[..., None], 0.0)
    lse = torch.where(total > 0, top + total.log(), float("inf"))
    t = torch.arange(q.shape[0], device="cuda")
    req = torch.searchsorted(cu, t, right=True) - 1
    mine = (req, t - cu[req])
    return o[mine].to(torch.bfloat16), lse[mine], top[mine]


def _verify_plain(s):
    """The nodes in index order: a node is tested when its parent is the last one kept.  r, what is left of the
    target's row after the rejections at a node, is rounded to 32 bits; its sums are taken in 64."""
    cu, p_rows, q_rows, vocab = s["cu_seqlens_q"].long(), s["target_probs"], s["draft_probs"], s["vocab"]
    up, token, u = _padded(s, s["parents"], -2), _padded(s, s["tokens"].long(), 0), _padded(s, s["accept_u"], 2.0)
    n_req, reqs = up.shape[0], torch.arange(up.shape[0], device="cuda")
    cur, kept = torch.zeros(n_req, dtype=torch.long, device="cuda"), torch.ones(n_req, dtype=torch.long, device="cuda")
    left = p_rows[cu[:-1]]                                             # r of the current node
    taken = torch.zeros(n_req, device="cuda")                          # C
    mass = torch.ones(n_req, dtype=torch.float64, device="cuda")       # Z
    keep = torch.full((n_req, s["max_keep"] + 1), -1, dtype=torch.long, device="cuda")
    out = keep.clone()
    keep[:, 0] = 0
    for c in range(1, s["max_n"]):
        x, asked = token[:, c], (up[:, c] == cur) & (kept < s["max_keep"])
        r = left[reqs, x].double()
        q = 1.0 if q_rows is None else q_rows[cu[:-1] + cur, x].double()
        yes = asked & (u[:, c].double() * q * mass < r)
        no = asked & ~yes
        at = torch.where(yes, kept, s["max_keep"])                     # the last column is thrown away
        keep[reqs, at] = c
        out[reqs, torch.where(yes, kept - 1, s["max_keep"])] = x
        cur, kept = torch.where(yes, c, cur), kept + yes
        row = cu[:-1] + cur
        if q_rows is None:
            mass = torch.where(no, mass - r, mass)
            left[reqs, x] = torch.where(no, 0.0, left[reqs, x])
        else:
            taken = torch.where(no, (taken + mass).float(), taken)
            less = (p_rows[row].double() - taken.double()[:, None] * q_rows[row].double()).clamp(min=0).float()
            left = torch.where(no[:, None], less, left)
            mass = torch.where(no, left.double().sum(-1), mass)
        left = torch.where(yes[:, None], p_rows[row], left)
        taken, mass = torch.where(yes, 0.0, taken), torch.where(yes, 1.0, mass)
    left = torch.where((left.amax(-1) > 0)[:, None], left, p_rows[cu[:-1] + cur])
    sums = left.double().cumsum(-1)
    new = (sums <= (s["sample_u"].double() * sums[:, -1])[:, None]).sum(-1)
    last = torch.where(left > 0, torch.arange(vocab, device="cuda"), -1).amax(-1)
    out[reqs, kept - 1] = torch.minimum(new, last)
    cut = slice(0, s["max_keep"])
    return dict(keep=keep[:, cut].int(), out_tokens=out[:, cut].int(), n_keep=kept.int())


def _commit_plain(s):
    pool, page, table, keep = s["kv_pool"], s["page"], s["block_table"].long(), s["keep"].long()
    cu, n_k, width = s["cu_seqlens_q"].long(), s["seqlens_k"].long(), s["block_table"].shape[1]
    before, done = n_k - (cu[1:] - cu[:-1]), s["n_keep"] < 0
    kept = s["n_keep"].clamp(min=0).long()
    i = torch.arange(keep.shape[1], device="cuda")
    moves = i < kept[:, None]

    def rows(pos):                        # what is not moved writes the first new row to itself
        pos = torch.where(moves, before[:, None] + pos, before[:, None])
        return (table.gather(1, pos // page) * page + pos % page).flatten()

    pool[:, rows(i)] = pool[:, rows(keep)]
    length = torch.where(done, 0, before + kept)
    first, last = (length + page - 1) // page, (n_k + page - 1) // page
    start, n_free = s["free_start"].long()[0], s["free_pages"].shape[0]
    back = last - first
    ahead = back.cumsum(0) - back
    col = torch.arange(width, device="cuda")
    freed = (col >= first[:, None]) & (col < last[:, None])
    place = torch.where(freed, start - 1 - (ahead[:, None] + col - first[:, None]), n_free)
    spare = torch.cat([s["free_pages"], s["free_pages"][:1]])
    spare[place.flatten()] = s["block_table"].flatten()
    s["free_pages"].copy_(spare[:n_free])
    counts = torch.stack([kept.sum(), start - back.sum(), torch.zeros_like(start)])
    return dict(kv_pool=pool, seqlens=length.int(), counts=counts.int(), free_pages=s["free_pages"])


def run(s):
    if own:
        import sparse_mla_attention_fwd_gb300 as smla
        if s["op"] == "plan":
            mask, positions = smla.sparse_mla_plan_tree(s["parents"], s["cu_seqlens_q"], s["seqlens_k"], s["words"])
            return dict(tree_mask=mask, positions=positions)
        if s["op"] == "attention":
            return smla.sparse_mla_tree_fwd_paged(s["q"], s["kv_pool"], s["block_table"], s["cu_seqlens_q"], s["seqlens_k"],
                                                  s["tree_mask"], page_block=s["page"], attn_sink=s["attn_sink"])
        if s["op"] == "verify":
            keep, out, n_keep = smla.sparse_mla_verify_tree(s["target_probs"], s["tokens"], s["parents"], s["cu_seqlens_q"],
                                                            s["accept_u"], s["sample_u"], s["max_keep"],
                                                            draft_probs=s["draft_probs"])
            return dict(keep=keep, out_tokens=out, n_keep=n_keep)
        seqlens, counts = smla.sparse_mla_commit_tree(s["keep"], s["n_keep"], s["cu_seqlens_q"], s["seqlens_k"],
                                                      s["block_table"], s["kv_pool"], page_block=s["page"],
                                                      free_pages=s["free_pages"], free_start=s["free_start"])
        return dict(kv_pool=s["kv_pool"], seqlens=seqlens, counts=counts, free_pages=s["free_pages"])
    return {"plan": _plan_plain, "attention": _attention_plain, "verify": _verify_plain, "commit": _commit_plain}[s["op"]](s)


# ------------------------------------------------------------------------- what has to be done
def work(case):
    n, k = _sizes(case)
    rows, words = sum(n), -(-case["n_max"] // 32)
    if case["op"] == "plan":
        rows += case["pad"]
        return dict(bytes=rows * (8 + 4 * words) + len(n) * 8 + 4, flops=0)
    if case["op"] == "verify":
        # the row that the last token is drawn from, and the draft's row where a draft was rejected: about six in ten of the
        # drafts are kept
        vocab = case["vocab"]
        less = sum(1 - 0.6 ** (m - 1) for m in n) if case["probs"] else 0
        return dict(bytes=int((len(n) + less) * vocab * 4) + len(n) * (8 + 8 * max(n)) + rows * (20 if case["probs"] else 16),
                    flops=int((len(n) + 2 * less) * vocab))
    if case["op"] == "commit":
        # kept rows that are not in their place yet: the first is, a kept path of the drawn length moves nearly all others
        moved = sum((min(m, case["n_max"], 9) - 1) / 2 for m in n) * 0.95
        page = case["page"]
        return dict(bytes=int(moved * case["layers"] * case["d_qk"] * 4) + len(n) * (16 + 4 * min(case["n_max"], 9)) + 16, flops=0)
    heads, d = case["heads"], case["d_qk"]
    pairs = sum(m * (x - m) for m, x in zip(n, k)) + rows     # the prefix, and a token at least itself
    return dict(bytes=sum(k) * d * 2 + rows * heads * ((d + D_V) * 2 + 8) + rows * words * 4 + sum(-(-x // case["page"]) for x in k) * 4,
                flops=pairs * heads * 2 * (d + D_V))


# ---------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The attention, request by request; the bits of a mask word are looked at one by one."""
    if case["op"] != "attention" or work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    q, cu, page = s["q"], s["cu_seqlens_q"].tolist(), s["page"]
    out = torch.zeros(q.shape[0], q.shape[1], D_V, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], float("inf"), dtype=torch.float64, device="cuda")
    top = torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
    masks = [[word & 0xffffffff for word in row] for row in s["tree_mask"].tolist()]
    for b, n_k in enumerate(s["seqlens_k"].tolist()):
        t0, t1 = cu[b], cu[b + 1]
        pages = s["block_table"][b, :-(-n_k // page)].long()
        kv = s["kv_pool"].reshape(-1, page, q.shape[2])[pages].reshape(-1, q.shape[2])[:n_k].double()
        hidden = torch.tensor([[not masks[t][j // 32] >> (j % 32) & 1 for j in range(t1 - t0)] for t in range(t0, t1)], device="cuda")
        for a in range(t0, t1, 16):
            e = min(a + 16, t1)
            z = torch.einsum("thd,kd->thk", q[a:e].double(), kv) / q.shape[2] ** 0.5
            z[..., n_k - (t1 - t0):] += torch.where(hidden[a - t0:e - t0], float("-inf"), 0.0)[:, None]
            top[a:e] = z.max(-1).values
            lse[a:e] = torch.logsumexp(z, -1)
            full = lse[a:e] if s["attn_sink"] is None else torch.logaddexp(lse[a:e], s["attn_sink"].double()[None, :])
            out[a:e] = torch.einsum("thk,kd->thd", (z - full[..., None]).exp(), kv[:, :D_V])
    return out, lse, top
