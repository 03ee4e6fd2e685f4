"""The cases of perf/more_operators.py through the framework: the attention against its 64-bit values, the other operators
equal to their plain forms; every listed case, and seeded ones from the ranges that those stand for."""
import random

import pytest
import torch

from perf import more_operators as operators

pytestmark = pytest.mark.gpu

U16, U32 = 2.0 ** -8, 2.0 ** -24
SEED = 7


def drawn(n, most_flops):
    rng, out = random.Random(2025), []
    while len(out) < n:
        case = operators.draw(rng)
        if operators.work(case)["flops"] <= most_flops:   # 64-bit products of the larger ones take too long here
            out.append(case)
    return out


CASES = operators.listed() + drawn(14, 5e11)


@pytest.fixture(autouse=True)
def device_status():
    yield
    torch.cuda.synchronize()
    import sparse_mla_attention_fwd_gb300 as smla
    assert smla.sparse_mla_device_status() == 0


def through_the_framework(monkeypatch, case):
    state = operators.prepare(case, SEED)
    monkeypatch.setattr(operators, "own", True)
    got = operators.run(state)
    monkeypatch.setattr(operators, "own", False)
    return state, got


def check_equal(monkeypatch, case):
    want = operators.run(operators.prepare(case, SEED))
    _, got = through_the_framework(monkeypatch, case)
    assert got.keys() == want.keys()
    for name in want:
        assert torch.equal(got[name], want[name]), name


def check_attention(monkeypatch, case):
    s, (out, lse, top) = through_the_framework(monkeypatch, case)
    o, z, m = operators.exact(case, SEED)
    d, longest = case["d_qk"], case["kv_max"]
    q_norm, k_norm = s["q"].float().norm(dim=-1).max(), s["kv_pool"].float().norm(dim=-1).max()
    v_norm = float(s["kv_pool"][..., :512].float().norm(dim=-1).max())
    # fp32 sums of d products: d 2^-23 of the sum of magnitudes, which is at most |q| |k|
    ds = float(q_norm * k_norm) * d ** -0.5 * d * 2 * U32
    live = torch.isfinite(z)
    assert bool((lse[~live] == z[~live].float()).all()) and bool((top[~live] == m[~live].float()).all())
    assert float((top.double() - m)[live].abs().max()) <= ds + 4 * U32 * float(m[live].abs().max())
    assert float((lse.double() - z)[live].abs().max()) <= ds + (longest + 16) * U32 + 8 * U32 * (1 + float(z[live].abs().max()))
    # out, every row: each weight is off by at most a rounding to bf16 and its logit's error, which is at most that part of
    # the largest |v|; then its own rounding
    err, size = (out.double() - o).norm(dim=-1), o.norm(dim=-1)
    worst = v_norm * (U16 + 2.1 * ds + 2 * (longest + 16) * U32) * (1 + U16) + size * U16 + 1e-30
    assert bool((err <= worst).all())
    # over all rows: the roundings of weights of independent rows of V add up as their squares do, to at most 2^-8 of |out| in
    # the mean, and so does the output's own: sqrt(2) 2^-8 together
    assert float(err.norm() / size.norm()) <= 1.5 * U16


@pytest.mark.parametrize("case", CASES, ids=lambda c: c.get("name") or "drawn " + c["op"])
def test_case(monkeypatch, case):
    (check_attention if case["op"] == "attention" else check_equal)(monkeypatch, case)
