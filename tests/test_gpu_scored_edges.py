"""Scored decode, selection and what they share with the other calls, at the edges: request ids that
are used again, sums of many kv heads, rows of more keys than shared memory holds, capture of a
decode, outputs on another stream, the statistics of the last decode."""
import numpy as np
import pytest

from attend_ref import SCALE
from test_gpu_attend import MMA, Pool, kvq, mixed, rand  # noqa: F401
from test_gpu_scored import check_select, step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("first", [True, False])
def test_a_request_id_used_again_without_pages(kvq, lists, first):
    """A request closed and opened again, empty or with list tokens only, next to one with pages: its
    rows of scores stay, and so does what lies around them (the earlier request had more positions
    than a row holds)."""
    P = Pool(kvq, 2, [mixed(500, 2), mixed(70, 1)] if first else [mixed(70, 1), mixed(500, 2)], seed=7)
    pool, r = P.pool, 0 if first else 1
    flat = torch.rand(2 * 2 * 70 + 8192, device="cuda", generator=P.gen)
    kept = flat.clone()
    scores = flat[4096:4096 + 280].view(2, 2, 70)
    pool.close_request(P.ids[r])
    assert pool.open() == P.ids[r]
    P.widths[r] = []
    fp = None
    if lists:
        pool.fp_configure(20)
        k, v = rand((9, 2, 128), P.gen), rand((9, 2, 128), P.gen)
        pool.fp_append(P.ids[r], k, v)
        fp = {r: k.double().cpu().numpy()}
    for _ in range(2):
        step(P, 8, scores, 0.5, fp=fp)
    assert torch.equal(scores[r], kept[4096:4096 + 280].view(2, 2, 70)[r])
    assert torch.equal(flat[:4096], kept[:4096]) and torch.equal(flat[4376:], kept[4376:])
    for per_head in (False, True):
        got = check_select(P, scores, 30, 0, per_head)
        assert (got[r] == -1).all()
    # the id in use again, with fewer tokens than before
    w = mixed(45, 3)
    pool.append(rand((45, 2, 128), P.gen), rand((45, 2, 128), P.gen), [P.ids[r]] * 45, w)
    P.widths[r] = list(map(int, w))
    step(P, 8, scores, 1.0, fp=fp)
    check_select(P, scores, 30, 3, False)
