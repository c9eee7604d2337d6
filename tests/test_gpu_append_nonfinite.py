"""New tokens whose indexer key holds an infinity or a NaN: a NaN scale and zero codes in every form
of the append, scores that are NaN for that key alone, and a selection that takes it."""
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


def _keys(rows, d):
    """Keys and the rows that are not finite."""
    g = torch.Generator(device="cuda").manual_seed(71)
    k = torch.randn(rows, d["d_idx"], generator=g, device="cuda")
    k[0, 3] = float("nan")
    k[1, d["d_idx"] - 1] = float("inf")
    k[2, 0] = float("-inf")
    k[3] = float("nan")
    k[4].view(torch.int32)[5] = -1                   # a NaN with its sign set
    k[5] = 3.0e38                                    # finite, the largest scales
    k[6] = 0
    return k, [0, 1, 2, 3, 4]


@pytest.mark.parametrize("layout", ["paged", "contiguous", "interleaved"])
@pytest.mark.parametrize("d", [FULL, TINY], ids=["full", "tiny"])
@pytest.mark.parametrize("mode", ["decode", "chunk"])
@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
def test_non_finite_keys(dsa, q8, mode, d, layout):
    new, ctx = ([1] * 9, [70 + i for i in range(9)]) if mode == "decode" else ([5, 4], [300, 64])
    pg = Pages(new, ctx, paged=layout != "contiguous", seed=53)
    pb = pg.problem(dsa, d, 64, mode)
    k_new, bad = _keys(pg.rows, d)
    kv_new = ref.latents(pg.rows, d, 72)
    rb = ref.row_bytes(d) if q8 else 2 * d["d_qk"]
    kv = torch.zeros(pg.kv_rows, rb, dtype=torch.uint8, device="cuda")
    if layout == "interleaved":
        k8, ks = torch.full((pg.kv_rows // 64, 64 * (d["d_idx"] + 4)), 7, dtype=torch.uint8,
                            device="cuda"), None
    else:
        k8 = torch.full((pg.kv_rows, d["d_idx"]), 7, dtype=torch.uint8, device="cuda")
        ks = torch.full((pg.kv_rows,), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = dsa.dsa_cache_append_q8 if q8 else dsa.dsa_cache_append
    assert call(pb, k_new, kv_new, k8, ks, kv, status) == dsa.DSA_OK
    assert int(status.item()) == 0
    good = [r for r in range(pg.rows) if r not in bad]
    codes, scale = ref.key_codes(k_new[good].cpu().numpy())
    for r in range(pg.rows):
        at = int(pg.phys(*pg.row(r)).reshape(-1)[0]) if mode == "chunk" else int(
            pg.phys(r, [ctx[r] - 1])[0])
        if ks is None:
            page, j = to_np(k8[at // 64]), at % 64
            c = page[j * d["d_idx"]:(j + 1) * d["d_idx"]]
            s = page[64 * d["d_idx"]:].view(np.float32)[j]
        else:
            c, s = to_np(k8[at]), to_np(ks[at])
        if r in bad:
            assert np.isnan(s) and not c.any(), r
        else:
            i = good.index(r)
            assert np.array_equal(c, codes[i]) and s == scale[i], r


@pytest.mark.parametrize("mode", ["decode", "chunk"])
def test_scores_and_selection_of_a_non_finite_key(dsa, mode):
    d, topk = FULL, 64
    new, ctx = ([1, 1], [500, 300]) if mode == "decode" else ([3, 2], [500, 300])
    pg = Pages(new, ctx, seed=54)
    pb = pg.problem(dsa, d, topk, mode)
    qi, qs, w, k8, ks = ref.indexer_inputs(pg.rows, pg.kv_rows, d, 73)
    k_new = torch.randn(pg.rows, d["d_idx"], device="cuda")
    k_new[0, 7] = float("nan")                       # the first new token of sequence 0
    kv_new = ref.latents(pg.rows, d, 74)
    kv8 = torch.from_numpy(ref.pack_rows(ref.latents(pg.kv_rows, d, 75), d)).cuda()
    assert dsa.dsa_cache_append_q8(pb, k_new, kv_new, k8, ks, kv8) == dsa.DSA_OK
    q = (torch.randn(pg.rows, d["h"], d["d_qk"], device="cuda")).to(torch.bfloat16)
    n = dsa.dsa_forward_q8_workspace_size(pb)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    idx = torch.full((pg.rows, topk), -7, dtype=torch.int32, device="cuda")
    sel = torch.zeros(pg.rows, topk, device="cuda")
    out = torch.empty(pg.rows, d["h"], d["d_v"], dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(pg.rows, d["h"], device="cuda")
    assert dsa.dsa_forward_q8(pb, qi, qs, w, k8, ks, q, kv8, idx, out, lse, ws, n,
                              sel_out=sel) == dsa.DSA_OK
    key = ctx[0] - new[0]                            # its position, seen by the rows of sequence 0
    for r in range(pg.rows):
        row, s = to_np(idx[r]), to_np(sel[r])
        assert (np.diff(row) > 0).all() and row[0] >= 0
        if r < new[0]:
            assert key in row and np.isnan(s[row == key]).all() and np.isnan(s).sum() == 1
        else:
            assert not np.isnan(s).any()
    values = torch.from_numpy(ref.unpack_rows(kv8.cpu().numpy(), d)).cuda()
    geo = pg if mode == "chunk" else Pages([1, 1], ctx, seed=54)
    ref.check_attention_rows(out, lse, q, values, idx, geo, d["d_qk"] ** -0.5, d)
