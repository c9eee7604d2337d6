"""Attention over every prior key at the longest context it takes, split and in one piece."""
import pytest
import torch

from tests import paged_ref as ref
from tests.paged_ref import FULL, Pages
from tests.test_gpu_paged_q8 import _attend, _cache, _queries, dsa  # noqa: F401

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
@pytest.mark.parametrize("rows", [2, 150])
def test_every_key_at_the_limit(dsa, q8, rows):  # noqa: F811
    d = FULL
    pg = Pages([rows], [131072], seed=61)
    pb = pg.problem(dsa, d, 2048)
    cache, values = _cache(pg, d, q8, 401)
    q = _queries(rows, d, 402)
    out, lse, status = _attend(dsa, pb, q8, q, cache, None, rows)
    assert status == 0
    ref.check_attention_rows(out, lse, q, values, None, pg, d["d_qk"] ** -0.5, d,
                             rows=[0, rows - 1])
