"""The selection over rows whose scores hold NaN and infinities: a NaN ranks with +infinity (the
smaller index first), and every entry of every row is written."""
import numpy as np
import pytest
import torch

from tests import paged_ref as ref
from tests.paged_ref import FULL, TINY, Pages
from tests.parity import to_np

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_long_04_b200 as m
    return m


def _expect(scores, k):
    s = np.where(np.isnan(scores), np.float32(np.inf), scores).astype(np.float64)
    pick = np.sort(np.lexsort((np.arange(len(s)), -s))[:k])
    return np.concatenate([pick, np.full(k - len(pick), -1)]).astype(np.int32)


def _poison(slab):
    """Rows 0, 1, ..: a few NaN; NaN of the other sign; as many NaN as are taken and more; NaN alone;
    NaN among infinities of both signs; -inf alone; NaN among equal scores."""
    n = slab.shape[1]
    g = torch.Generator(device="cuda").manual_seed(3)
    pick = lambda m: torch.randperm(n, generator=g, device="cuda")[:m]
    bits = slab.view(torch.int32)
    slab[0, pick(3)] = float("nan")
    bits[1, pick(5)] = -1                            # sign bit set, 0xFFFFFFFF
    bits[1, pick(5)] = 0x7F800001
    slab[2, pick(n // 2)] = float("nan")
    slab[3] = float("nan")
    slab[4, pick(40)] = float("inf")
    slab[4, pick(40)] = float("nan")
    slab[4, pick(40)] = float("-inf")
    slab[5] = float("-inf")
    slab[6] = 1.0
    slab[6, pick(7)] = float("nan")


@pytest.mark.parametrize("mode", ["prefill", "decode", "chunk"])
@pytest.mark.parametrize("n,topk", [(700, 64), (5000, 2048), (70001, 2048), (2048, 2048)])
def test_nan_scores(dsa, mode, n, topk):
    rows = 8
    if mode == "prefill":                            # the last rows of one sequence
        pb = dsa.make_problem(mode="prefill", topk=topk, softmax_scale=0.04, num_kv_rows=n,
                              seqlens=[n], cu_seqlens=torch.tensor([0, n], dtype=torch.int32,
                                                                   device="cuda"), **FULL)
        first, seen = n - rows, [n - rows + i + 1 for i in range(rows)]
    else:
        new, ctx = ([1] * rows, [n] * rows) if mode == "decode" else ([rows], [n])
        pg = Pages(new, ctx, paged=mode == "chunk", seed=51)
        pb = pg.problem(dsa, FULL, topk, mode)
        first, seen = 0, [pg.row(r)[1] + 1 for r in range(rows)]
    ld = (n + 3) // 4 * 4
    slab = torch.randn(rows, ld, device="cuda")
    _poison(slab)
    got = to_np(slab)
    for with_hist in (False, True):
        hist = None
        if with_hist:                                # the counts that the indexer would make
            hist = torch.zeros(rows, 2048, dtype=torch.int32, device="cuda")
            for r in range(rows):
                s = np.where(np.isnan(got[r, :seen[r]]), np.float32(np.inf), got[r, :seen[r]]) + np.float32(0)
                u = s.view(np.uint32)
                key = np.where(u >> 31, ~u, u | np.uint32(0x80000000))
                hist[r] = torch.from_numpy(np.bincount(key >> 21, minlength=2048).astype(np.int32))
        idx = torch.full((rows, topk), -7, dtype=torch.int32, device="cuda")
        sel = torch.full((rows, topk), 9.0, device="cuda")
        assert dsa.dsa_topk(pb, slab, ld, first, rows, idx, hist=hist, sel_out=sel) == dsa.DSA_OK
        out, sv = to_np(idx), to_np(sel)
        for r in range(rows):
            want = _expect(got[r, :seen[r]], topk)
            assert np.array_equal(out[r], want), (r, with_hist)
            ok = want >= 0
            assert np.array_equal(sv[r, ok].view(np.uint32), got[r, want[ok]].view(np.uint32)), r
            assert not sv[r, ~ok].any()


@pytest.mark.parametrize("d,mode", [(FULL, "decode"), (FULL, "chunk"), (TINY, "chunk")],
                         ids=["full-decode", "full-chunk", "tiny-chunk"])
def test_keys_with_a_nan_scale(dsa, d, mode):
    """Keys whose scale is NaN score NaN for every row that sees them: the fused selection takes them
    first, then the largest of the others."""
    new, ctx = ([1] * 3, [900, 5000, 130]) if mode == "decode" else ([5, 1, 70], [900, 5000, 130])
    pg = Pages(new, ctx, seed=52)
    topk = 128
    pb = pg.problem(dsa, d, topk, mode)
    q8, qs, w, k8, ks = ref.indexer_inputs(pg.rows, pg.kv_rows, d, 61)
    bad = {0: [3, 700], 1: list(range(100, 400)), 2: [0, 64]}
    for b, keys in bad.items():
        ks[torch.as_tensor(pg.phys(b, keys), device="cuda")] = float("nan")
    n = dsa.dsa_indexer_topk_workspace_size(pb, pg.rows)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    idx = torch.full((pg.rows, topk), -7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert dsa.dsa_indexer_topk(pb, q8, qs, w, k8, ks, 0, pg.rows, idx, ws, n, status) == dsa.DSA_OK
    ld = (max(ctx) + 3) // 4 * 4
    slab = torch.zeros(pg.rows, ld, device="cuda")
    assert dsa.dsa_indexer_scores(pb, q8, qs, w, k8, ks, 0, pg.rows, slab, ld, status) == dsa.DSA_OK
    assert int(status.item()) == 0
    got, out = to_np(slab), to_np(idx)
    for r in range(pg.rows):
        b, pos = pg.row(r) if mode == "chunk" else (r, ctx[r] - 1)
        seen = [k for k in bad[b] if k <= pos]
        assert np.isnan(got[r, seen]).all()
        assert np.isnan(got[r, :pos + 1]).sum() == len(seen)
        assert np.array_equal(out[r], _expect(got[r, :pos + 1], topk)), r
