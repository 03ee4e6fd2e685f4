"""Verification at every choice of CTAs a request and loads under way that the number of requests leads to."""
import pytest
import torch

from test_tree_step_gpu import verify_case, verify_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("n_req", [36, 37, 49, 50, 57, 58, 72, 73, 110, 111, 114, 115, 152, 153, 228, 229, 304, 305, 456, 457])
def test_verify_at_each_launch_shape(n_req, draft):
    """The numbers of requests at which the rule changes on 152 SMs, with a vocabulary of several tiles a CTA: rows that lie alike for
    16-byte loads, and rows of the target and the draft that do not."""
    sizes = [1 + (7 * b + n_req) % 4 for b in range(n_req)]
    w = verify_case(n_req, sizes, 9001, draft, "star" if n_req % 2 else "tree", scale=2.0 if draft else 6.0, apart=1.5)
    kept = verify_check(w)[2]
    assert int(kept.max()) > 1 and int((kept == 1).sum()) > 0
    n = sum(sizes)
    for column, width in ((0, 9004), (3, 9009)):
        wide = torch.full((n, width), float("nan"), device="cuda")
        wide[:, column:column + 9001] = w["target_probs"]
        verify_check(dict(w, target_probs=wide[:, column:column + 9001]))


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("vocab", [1025, 1500, 2049, 3000, 4097, 5000])
def test_verify_with_few_ctas_a_request(vocab, draft):
    """Small vocabularies keep clusters small whatever the number of requests."""
    for n_req in (3, 73, 120):
        verify_check(verify_case(vocab + n_req, [1 + (5 * b) % 4 for b in range(n_req)], vocab, draft, "tree", apart=2.0))
