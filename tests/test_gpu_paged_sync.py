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


def _zeros(out, lse, rows):
    assert (out[rows] == 0).all() and (lse[rows] == float("-inf")).all()


@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
@pytest.mark.parametrize("d", [FULL, TINY], ids=["full", "tiny"])
def test_rows_without_keys_repeat_exactly(dsa, d, q8):  # noqa: F811
    """Rows whose entries are all -1, among rows with one key and rows with many, of many sequences:
    exact zeros and -inf every time."""
    pg = Pages([3, 1, 0, 4] * 60, [700, 1, 9, 2500] * 60, seed=42)
    pb = pg.problem(dsa, d, 128)
    cache, values = _cache(pg, d, q8, 311)
    q = _queries(pg.rows, d, 312)
    idx = torch.from_numpy(ref.random_selection(pg, 128, 313)).cuda()
    empty = torch.arange(pg.rows, device="cuda") % 3 != 0
    idx[empty] = -1
    idx[3::6, 1:] = -1                               # one key
    out, lse, status = _repeat(dsa, pb, q8, q, cache, idx, pg.rows, 150, d, Traffic())
    assert status == 0
    _zeros(out, lse, empty)
    ref.check_attention_rows(out, lse, q, values, idx, pg, d["d_qk"] ** -0.5, d,
                             rows=range(0, pg.rows, 9))


@pytest.mark.parametrize("mode,q8", [("decode", True), ("chunk", True), ("chunk", False)])
def test_splits_without_keys_repeat_exactly(dsa, mode, q8):  # noqa: F811
    """Few rows are split many ways by the longest possible context: contexts of 1, 70 and 300 keys
    leave most splits without a tile, a row without entries all of them."""
    d = FULL
    new, ctx = [1, 1, 1, 1], [1, 70, 300, 900]
    pg = Pages(new, ctx, seed=43, max_seqlen=100000)
    pb = pg.problem(dsa, d, 2048, mode)
    size = dsa.dsa_sparse_mla_q8_workspace_size if q8 else dsa.dsa_sparse_mla_workspace_size
    assert size(pb, 4) >= 8 * 4 * 128 * 513 * 4      # 8 splits at least; the contexts have 1, 2, 5 tiles
    cache, values = _cache(pg, d, q8, 321)
    q = _queries(pg.rows, d, 322)
    idx = torch.from_numpy(ref.random_selection(pg, 2048, 323)).cuda()
    idx[3] = -1
    out, lse, status = _repeat(dsa, pb, q8, q, cache, idx, pg.rows, 400, d, Traffic())
    assert status == 0
    _zeros(out, lse, [3])
    ref.check_attention_rows(out, lse, q, values, idx, pg, d["d_qk"] ** -0.5, d)


@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
def test_short_contexts_of_a_long_batch_repeat_exactly(dsa, q8):  # noqa: F811
    """The same without indices, and through the selection: the short contexts of a batch whose
    longest is 5000 keys."""
    d = FULL
    pg = Pages([1, 2, 1], [1, 40, 5000], seed=44)
    pb = pg.problem(dsa, d, 2048)
    cache, values = _cache(pg, d, q8, 331)
    q = _queries(pg.rows, d, 332)
    traffic = Traffic()
    out, lse, status = _repeat(dsa, pb, q8, q, cache, None, pg.rows, 100, d, traffic)
    assert status == 0
    ref.check_attention_rows(out, lse, q, values, None, pg, d["d_qk"] ** -0.5, d)
    qi, qs, w, k8, ks = ref.indexer_inputs(pg.rows, pg.kv_rows, d, 333)
    n = (dsa.dsa_forward_q8_workspace_size if q8 else dsa.dsa_forward_workspace_size)(pb)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    idx = torch.empty(pg.rows, 2048, dtype=torch.int32, device="cuda")
    forward = dsa.dsa_forward_q8 if q8 else dsa.dsa_forward
    first = None
    for _ in range(100):
        traffic.more()
        assert forward(pb, qi, qs, w, k8, ks, q, cache, idx, out, lse, ws, n) == dsa.DSA_OK
        torch.cuda.synchronize()
        if first is None:
            first = (idx.clone(), out.clone(), lse.clone())
            ref.check_attention_rows(out, lse, q, values, idx, pg, d["d_qk"] ** -0.5, d)
        for a, b in zip(first, (idx, out, lse)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("mode,q8", [("decode", True), ("chunk", True), ("chunk", False)])
@pytest.mark.parametrize("every", [True, False], ids=["every", "selected"])
def test_attention_sees_the_token_written_just_before(dsa, mode, q8, every):  # noqa: F811
    """Append and attention back to back, the same places overwritten step after step: each step
    reads the rows of its own append, as with the device idle in between."""
    d = FULL
    batch = 40
    new = [1] * batch if mode == "decode" else [1, 3] * (batch // 2)
    pg = Pages(new, [200 + 7 * b for b in range(batch)], seed=45)
    pb = pg.problem(dsa, d, 512, mode)
    cache, _ = _cache(pg, d, q8, 341)
    k8 = torch.zeros(pg.kv_rows, 128, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(pg.kv_rows, device="cuda")
    k_new = torch.randn(pg.rows, 128, device="cuda")
    q = _queries(pg.rows, d, 342)
    idx = None if every else torch.from_numpy(ref.random_selection(pg, 512, 343)).cuda()
    n = (dsa.dsa_sparse_mla_q8_workspace_size if q8 else dsa.dsa_sparse_mla_workspace_size)(
        pb, pg.rows)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    append = dsa.dsa_cache_append_q8 if q8 else dsa.dsa_cache_append
    attend = dsa.dsa_sparse_mla_fwd_q8 if q8 else dsa.dsa_sparse_mla_fwd
    steps = 12
    kv_new = [ref.latents(pg.rows, d, 350 + i) for i in range(steps)]
    runs = []
    for idle in (False, True):
        outs = [(torch.empty(pg.rows, d["h"], d["d_v"], dtype=torch.bfloat16, device="cuda"),
                 torch.empty(pg.rows, d["h"], device="cuda")) for _ in range(steps)]
        torch.cuda.synchronize()
        for x, (out, lse) in zip(kv_new, outs):
            assert append(pb, k_new, x, k8, ks, cache) == dsa.DSA_OK
            if idle:
                torch.cuda.synchronize()
            assert attend(pb, q, cache, idx, 0, pg.rows, out, lse, ws, n) == dsa.DSA_OK
        torch.cuda.synchronize()
        runs.append(outs)
    for (o, l), (oi, li) in zip(*runs):
        assert torch.equal(o, oi) and torch.equal(l, li)
    assert not torch.equal(runs[0][0][0], runs[0][1][0])
