"""The paged attention where its warps, and the two CTAs of a row, must wait for one another: calls
repeated many times, beside other traffic, give the same bits every time and the right ones."""
import numpy as np
import pytest
import torch

from tests import paged_ref as ref
from tests.paged_ref import FULL, TINY, Pages
from tests.test_gpu_paged_q8 import _attend, _cache, _queries, dsa  # noqa: F401

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


class Traffic:
    """Copies on another stream that take memory bandwidth and SMs from the calls beside them."""

    def __init__(self):
        self.stream = torch.cuda.Stream()
        self.a = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        self.b = torch.empty_like(self.a)
        torch.cuda.synchronize()

    def more(self):
        with torch.cuda.stream(self.stream):
            self.b.copy_(self.a)


def _repeat(dsa, pb, q8, q, cache, idx, rows, times, d, traffic):  # noqa: F811
    out, lse, status = _attend(dsa, pb, q8, q, cache, idx, rows, d=d)
    for _ in range(times):
        traffic.more()
        again, lagain, st = _attend(dsa, pb, q8, q, cache, idx, rows, d=d)
        assert st == status
        assert torch.equal(again, out) and torch.equal(lagain, lse)
    return out, lse, status


@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
@pytest.mark.parametrize("d", [FULL, TINY], ids=["full", "tiny"])
def test_logit_exchange_repeats_exactly(dsa, d, q8):  # noqa: F811
    """Rows of many tiles: a CTA overwrites its partner's logits of a tile with the next tile's only
    when the partner has read them."""
    pg = Pages([150, 60], [6000, 2300], seed=41)
    pb = pg.problem(dsa, d, 2048)
    cache, values = _cache(pg, d, q8, 301)
    q = _queries(pg.rows, d, 302)
    idx = torch.from_numpy(ref.random_selection(pg, 2048, 303)).cuda()
    out, lse, status = _repeat(dsa, pb, q8, q, cache, idx, pg.rows, 60, d, Traffic())
    assert status == 0
    ref.check_attention_rows(out, lse, q, values, idx, pg, d["d_qk"] ** -0.5, d,
                             rows=range(0, pg.rows, 11))
