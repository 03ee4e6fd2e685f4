"""Verification of drafted tokens where the decision is a near tie: random numbers next to the border of a comparison.

The plain loops decide in 64 bits.  A row's sum is at most 40 additions deep in the kernel (values of a tile, lanes, tiles,
warps, CTAs).  Each keeps its rounding in the second float, which is then at most 40 x 2^-24 of the sum and is itself rounded
to 24 bits at each of them: 40 x 41 / 2 x 2^-48 < 2^-38 of the sum in all.  Only cases with a margin above that are
tested; a comparison in plain fp32 errs by 2^-24 and fails a good part of them."""
import numpy as np
import pytest
import torch

from test_tree_step_gpu import verify_case, verify_check

pytestmark = pytest.mark.gpu

MARGIN = 2.0 ** -38
LAST = np.float32(1.0 - 2.0 ** -24)      # the largest number below 1


def rows_of(w, name):
    return w[name].cpu().numpy().astype(np.float64)


def next_to(x, rng):
    """fp32 numbers nearest to x or one further on either side, in [0, 1)."""
    near = x.astype(np.float32)
    side = rng.integers(-1, 2, x.shape)
    near = np.where(side < 0, np.nextafter(near, np.float32(0)), np.where(side > 0, np.nextafter(near, np.float32(2)), near))
    return np.clip(near, np.float32(0), LAST)


def residual(p, q, times):
    """What is left of p after so many rejections, its sum, and whether each rounding of C is clear of a tie."""
    C, Z, clear = np.zeros(len(p), dtype=np.float32), np.ones(len(p)), np.ones(len(p), dtype=bool)
    for _ in range(times):
        exact = C.astype(np.float64) + Z
        C = exact.astype(np.float32)
        half = np.spacing(C).astype(np.float64) / 2
        clear &= np.abs(np.abs(exact - C.astype(np.float64)) - half) > 4 * MARGIN
        r = np.maximum(p - C[:, None].astype(np.float64) * q, 0).astype(np.float32).astype(np.float64)
        Z = r.sum(1)
    return r, Z, clear


def rejected(seed, n_req, vocab, draft, times):
    """Stars whose first `times` children are turned down; the case, of each request r behind that and Z in 64 bits, and
    residual()'s last."""
    nodes = times + 2
    w = verify_case(seed, [nodes] * n_req, vocab, draft, kind="star", scale=1.0, apart=1.0)
    p = rows_of(w, "target_probs")[::nodes]
    tokens, u = w["tokens"].cpu().numpy().reshape(n_req, nodes), np.zeros((n_req, nodes), dtype=np.float32)
    u[:, 1:-1] = LAST
    every = np.arange(n_req)
    if draft:
        q = rows_of(w, "draft_probs")[::nodes]
        tokens[:, 1:-1] = (p / q).argmin(1)[:, None]
        r, Z, clear = residual(p, q, times)
    else:
        order = p.argsort(1)
        r, Z, clear = p.copy(), np.ones(n_req), np.ones(n_req, dtype=bool)
        for k in range(times):
            x = order[:, -1 - k]
            tokens[:, 1 + k] = x
            Z -= r[every, x]
            r[every, x] = 0
    return w, tokens, u, r, Z, clear


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("times", [1, 2, 3])
@pytest.mark.parametrize("vocab,n_req", [(300, 1500), (9001, 60)])
def test_accepts_next_to_the_border(vocab, n_req, times, draft):
    """u next to r(x) / (q(x) Z): kept exactly when u q(x) Z < r(x)."""
    w, tokens, u, r, Z, clear = rejected(31 + times, n_req, vocab, draft, times)
    rng, every = np.random.default_rng(times), np.arange(n_req)
    weight = (rows_of(w, "draft_probs")[::times + 2] if draft else np.ones_like(r)) * Z[:, None]
    fits = (r > 0) & (r < 0.9 * weight)
    assert fits.any(1).all()
    x = np.where(fits, rng.random(r.shape), -1).argmax(1)          # any token that may be kept and may be turned down
    tokens[:, -1] = x
    u[:, -1] = next_to(r[every, x] / weight[every, x], rng)
    off = np.abs(u[:, -1].astype(np.float64) * weight[every, x] - r[every, x]) / r[every, x]
    u[(off <= MARGIN) | ~clear, -1] = 0.5
    assert (off < 2.0 ** -23).sum() > n_req // 4                   # many are nearer than fp32 tells apart
    w["tokens"].copy_(torch.from_numpy(tokens.reshape(-1)))
    w["accept_u"].copy_(torch.from_numpy(u.reshape(-1)))
    kept = verify_check(w)[2]
    assert 0 < int((kept == 2).sum()) < n_req


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("times", [1, 2])
@pytest.mark.parametrize("vocab,n_req", [(300, 1500), (9001, 100), (50001, 6)])
def test_last_tokens_next_to_the_border(vocab, n_req, times, draft):
    """sample_u next to (r(0) + .. + r(v)) / sum r: the token is v or the one behind it."""
    w, tokens, u, r, _, clear = rejected(41 + times, n_req, vocab, draft, times)
    rng = np.random.default_rng(times)
    tokens[:, -1] = tokens[:, 1]                                   # turned down once more
    u[:, -1] = LAST
    if draft:      # the last rejection counts too
        p, q = rows_of(w, "target_probs")[::times + 2], rows_of(w, "draft_probs")[::times + 2]
        r, _, clear = residual(p, q, times + 1)
    sums = r.cumsum(1)
    total = sums[:, -1]
    v = rng.integers(vocab // 10, vocab - vocab // 10, n_req)
    s = next_to(sums[np.arange(n_req), v] / total, rng)
    off = np.abs(sums - (s.astype(np.float64) * total)[:, None]).min(1) / total
    s[(off <= MARGIN) | ~clear] = 0.5
    assert (off < 2.0 ** -23).sum() > n_req // 4
    w["tokens"].copy_(torch.from_numpy(tokens.reshape(-1)))
    w["accept_u"].copy_(torch.from_numpy(u.reshape(-1)))
    w["sample_u"].copy_(torch.from_numpy(s))
    assert bool((verify_check(w)[2] == 1).all())


@pytest.mark.parametrize("times", [1, 2, 4])
@pytest.mark.parametrize("vocab,n_req", [(50, 2000), (9001, 150)])
def test_residuals_against_the_rule_without_roundings(vocab, n_req, times):
    """r and C are rounded to fp32.  Against the rule in 64 bits throughout: C is off by its own rounding, 2^-24 of it, and by Z's
    error; r(v) by q(v) times that and its own rounding; Z by the sum of r's.  Where the decision's margin is larger, it is the same."""
    w, tokens, u, _, _, _ = rejected(51 + times, n_req, vocab, True, times)
    nodes, rng, every, half = times + 2, np.random.default_rng(vocab + times), np.arange(n_req), 2.0 ** -24
    p, q = rows_of(w, "target_probs")[::nodes], rows_of(w, "draft_probs")[::nodes]

    def exact(rejections):
        C, Z, off_c, off_z = np.zeros(n_req), np.ones(n_req), np.zeros(n_req), np.zeros(n_req)
        for k in range(rejections):
            C = C + Z
            off_c = off_c + off_z + (half * C if k else 0)         # the first sum is 1, which has no rounding
            r = np.maximum(p - C[:, None] * q, 0)
            Z = r.sum(1)
            off_z = off_c * q.sum(1) + half * Z
        return r, Z, off_c, off_z

    r, Z, off_c, off_z = exact(times)
    x, last = tokens[:, -1], rng.random(n_req).astype(np.float32)
    u[:, -1] = last
    left, need = last * q[every, x] * Z, r[every, x]
    clear = np.abs(left - need) > 1.01 * (last * q[every, x] * off_z + off_c * q[every, x] + half * need)
    clear |= (need == 0) & (p[every, x] < 0.99 * q[every, x])      # 0 with and without roundings
    kept = left < need
    r, Z, off_c, off_z = exact(times + 1)
    s = rng.random(n_req).astype(np.float32)
    sums = r.cumsum(1)
    drawn = (sums > (s * Z)[:, None]).argmax(1)
    sure = clear & (np.abs(sums - (s * Z)[:, None]).min(1) > 1.01 * (1 + s) * off_z)
    w["tokens"].copy_(torch.from_numpy(tokens.reshape(-1)))
    w["accept_u"].copy_(torch.from_numpy(u.reshape(-1)))
    w["sample_u"].copy_(torch.from_numpy(s))
    _, out, n_keep = (t.cpu().numpy() for t in verify_check(w))
    assert clear.mean() > 0.9 and sure.mean() > 0.3 and 0 < kept.sum() < n_req
    assert np.array_equal(n_keep[clear], 1 + kept[clear])
    again = sure & ~kept
    assert np.array_equal(out[again, 0], drawn[again])
