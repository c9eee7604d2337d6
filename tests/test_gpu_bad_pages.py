"""Pages outside the caches, whole or in part: their keys score 0, the other keys as without the bad
page, and no new token is written there."""
import numpy as np
import pytest
import torch

from tests import paged_ref as ref
from tests.paged_ref import FULL, TINY, Pages
from tests.parity import check_scores, to_np

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_long_04_b200 as m
    return m


@pytest.mark.parametrize("d,mode,layout", [
    (FULL, "decode", "paged"), (FULL, "decode", "interleaved"), (FULL, "chunk", "paged"),
    (FULL, "chunk", "interleaved"), (TINY, "chunk", "paged"), (TINY, "chunk", "interleaved")])
def test_scores_of_a_bad_page_are_zero(dsa, d, mode, layout):
    new, ctx = ([1, 1, 1], [2000, 700, 130]) if mode == "decode" else ([3, 70, 1], [2000, 700, 130])
    pg = Pages(new, ctx, seed=81)
    pb = pg.problem(dsa, d, 64, mode)
    q8, qs, w, k8, ks = ref.indexer_inputs(pg.rows, pg.kv_rows, d, 82)
    kin, sin = (ref.interleave(k8, ks), None) if layout == "interleaved" else (k8, ks)
    ld = (max(ctx) + 3) // 4 * 4
    good, status = torch.full((pg.rows, ld), -7.0, device="cuda"), torch.zeros(
        1, dtype=torch.int32, device="cuda")
    assert dsa.dsa_indexer_scores(pb, q8, qs, w, kin, sin, 0, pg.rows, good, ld,
                                  status) == dsa.DSA_OK
    assert int(status.item()) == 0
    bad = {0: [(3, -1), (20, pg.kv_rows // 64)], 1: [(10, 1 << 25)], 2: []}
    if layout == "paged":                           # a page of which the caches hold 40 rows
        pg.kv_rows -= 24
        pb = pg.problem(dsa, d, 64, mode)
        last = np.argwhere(pg.table == pg.kv_rows // 64)
        for b, j in last:
            if j * 64 < ctx[b]:
                bad[int(b)].append((int(j), pg.kv_rows // 64))
    for b, pages in bad.items():
        for j, page in pages:
            pg.d_table[b, j] = page
    slab = torch.full((pg.rows, ld), -7.0, device="cuda")
    for _ in range(2):
        status.zero_()
        assert dsa.dsa_indexer_scores(pb, q8, qs, w, kin, sin, 0, pg.rows, slab, ld,
                                      status) == dsa.DSA_OK
        assert int(status.item()) == dsa.DSA_DEVICE_BAD_INDEX
        for r in range(pg.rows):
            b, pos = pg.row(r) if mode == "chunk" else (r, ctx[r] - 1)
            want = good[r].clone()
            for j, _ in bad[b]:
                want[j * 64:min((j + 1) * 64, pos + 1)] = 0
            assert torch.equal(slab[r], want), r


@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
@pytest.mark.parametrize("mode", ["decode", "chunk"])
def test_append_into_a_page_in_part_outside(dsa, q8, mode):
    """A page of which the caches hold only the first rows takes no token in either mode (the indexer
    would not read it)."""
    d = FULL
    new, ctx = ([1, 1], [100, 70]) if mode == "decode" else ([2, 3], [100, 70])
    pg = Pages(new, ctx, seed=83, spare=0)
    pg.table[:, :2] = [[0, 3], [1, 2]]              # the last page under sequence 0's new tokens
    pg.d_table.copy_(torch.from_numpy(pg.table))
    rows = pg.kv_rows
    pg.kv_rows -= 4                                 # the last page holds 60 rows
    pb = pg.problem(dsa, d, 64, mode)
    rb = ref.row_bytes(d) if q8 else 2 * d["d_qk"]
    kv = torch.full((rows, rb), 7, dtype=torch.uint8, device="cuda")
    k8 = torch.full((rows, d["d_idx"]), 7, dtype=torch.uint8, device="cuda")
    ks = torch.full((rows,), 7.0, device="cuda")
    k_new = torch.randn(pg.rows, d["d_idx"], device="cuda")
    kv_new = ref.latents(pg.rows, d, 84)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = dsa.dsa_cache_append_q8 if q8 else dsa.dsa_cache_append
    assert call(pb, k_new, kv_new, k8, ks, kv, status) == dsa.DSA_OK
    assert int(status.item()) == dsa.DSA_DEVICE_BAD_INDEX
    want = {int(x) for x in pg.phys(1, np.arange(ctx[1] - new[1], ctx[1]))}
    assert set(np.nonzero(to_np(ks) != 7.0)[0].tolist()) == want
    assert set(np.nonzero((to_np(kv) != 7).any(axis=1))[0].tolist()) <= want
