"""The paged operators on the GPU against their 64-bit definitions (tests/paged_ref.py): the 8-bit
latent cache written and read back bit for bit, attention of single tokens and chunks over the
8-bit and bf16 caches, the chunk mode of the indexer and the top-k, and the whole path."""
import math

import numpy as np
import pytest
import torch

import oracle
from tests import paged_ref as ref
from tests.paged_ref import FULL, TINY, Pages
from tests.parity import check_scores, check_topk_exact, to_np

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_long_04_b200 as m
    return m


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _u8(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------------------- write

def _new_tokens(rows, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(rows, d["d_idx"], generator=g, device="cuda") * 3
    kv = ref.latents(rows, d, seed + 1)
    if rows > 8:
        k[1] = 0
        kv[1] = 0
        kv[2, :128] = 3.0e38                    # above 448 * 2^119: saturates
        kv[3, :128] = 1.0e-38                   # below the smallest scale
        kv[4, 5] = float("inf")
        kv[5, 127] = float("nan")
        # every half step of a binade against a scale of 1: ties to even
        kv[6, :128] = (torch.arange(128, device="cuda") / 16 + 1).to(torch.bfloat16)
        kv[6, 0] = 448.0
        kv[7, :128] = torch.linspace(-0.02, 0.02, 128, device="cuda").to(torch.bfloat16)
        kv[7, 1] = -256.0                       # codes reach the subnormals
        kv[8, d["d_v"]:] = float("inf")         # rotary dims are copied whatever they hold
    return k, kv


GEOMETRIES = [
    ("decode", [1] * 9, [700, 64, 1, 130, 4096, 65, 2, 63, 128]),
    ("decode", [1], [1]),
    ("chunk", [5, 0, 64, 1, 200], [5, 77, 130, 4000, 333]),
    ("chunk", [0, 33, 0], [9, 33, 1]),
]


@pytest.mark.parametrize("mode,new,ctx", GEOMETRIES)
@pytest.mark.parametrize("d", [FULL, TINY], ids=["full", "tiny"])
@pytest.mark.parametrize("layout", ["paged", "contiguous", "interleaved"])
@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
def test_append_bytes(dsa, mode, new, ctx, d, layout, q8):
    """Every byte of the caches: the new tokens' rows from the definition, all others as they
    were."""
    pg = Pages(new, ctx, paged=layout != "contiguous", seed=1)
    pb = pg.problem(dsa, d, 64, mode)
    g = torch.Generator(device="cuda").manual_seed(5)
    byte = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)
    rb = ref.row_bytes(d) if q8 else 2 * d["d_qk"]
    kv = byte(pg.kv_rows, rb)
    if layout == "interleaved":
        k8, ks = byte(pg.kv_rows // 64, 64 * (d["d_idx"] + 4)), None
    else:
        k8, ks = byte(pg.kv_rows, d["d_idx"]), torch.rand(pg.kv_rows, device="cuda")
    want_kv, want_k = kv.cpu().numpy().copy(), k8.cpu().numpy().copy()
    want_s = None if ks is None else ks.cpu().numpy().copy()
    k_new, kv_new = _new_tokens(pg.rows, d, 11)
    status = _status()
    if q8:
        st = dsa.dsa_cache_append_q8(pb, k_new, kv_new, k8, ks, kv, status)
    else:
        st = dsa.dsa_cache_append(pb, k_new, kv_new, k8, ks, kv, status)
    assert st == dsa.DSA_OK
    assert int(status.item()) == 0
    codes, scale = ref.key_codes(k_new.cpu().numpy())
    rows = (ref.pack_rows(kv_new, d) if q8 else kv_new.cpu().view(torch.int16).numpy().view(np.uint8))
    for r in range(pg.rows):
        b, pos = pg.row(r)
        at = int(pg.phys(b, [pos])[0])
        want_kv[at] = rows[r]
        if ks is not None:
            want_k[at], want_s[at] = codes[r], scale[r]
        else:
            page, j = at // 64, at % 64
            want_k[page, j * d["d_idx"]:(j + 1) * d["d_idx"]] = codes[r]
            s0 = 64 * d["d_idx"] + 4 * j
            want_k[page, s0:s0 + 4] = scale[r:r + 1].view(np.uint8)
    got = kv.cpu().numpy()
    if q8:                                       # a NaN scale may be any NaN
        dv, g4 = d["d_v"], 4 * (d["d_v"] // 128)
        a = np.ascontiguousarray(got[:, dv:dv + g4]).view(np.float32)
        w = np.ascontiguousarray(want_kv[:, dv:dv + g4]).view(np.float32)
        nan = np.repeat(np.isnan(a) & np.isnan(w), 4, axis=1)
        got[:, dv:dv + g4][nan] = want_kv[:, dv:dv + g4][nan] = 0
    assert np.array_equal(got, want_kv)
    assert np.array_equal(k8.cpu().numpy(), want_k)
    if ks is not None:
        assert np.array_equal(ks.cpu().numpy(), want_s)


@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
def test_append_skips_bad_entries(dsa, q8):
    """A page outside the caches, a context above max_seqlen, more new tokens than context: those
    tokens are skipped and reported, the others written."""
    d = FULL
    pg = Pages([3, 70, 4, 2], [300, 130, 64, 90], seed=2)
    pg.d_table[1, 1] = -1                        # positions 64..127 of sequence 1
    pg.d_table[1, 2] = pg.kv_rows // 64          # positions 128, 129
    pg.d_ctx[2] = pg.max_seqlen + 1
    pg.d_ctx[3] = 1                              # two new tokens, one cached
    pb = pg.problem(dsa, d, 64)
    rb = ref.row_bytes(d) if q8 else 2 * d["d_qk"]
    kv = torch.full((pg.kv_rows, rb), 7, dtype=torch.uint8, device="cuda")
    k8 = torch.full((pg.kv_rows, 128), 7, dtype=torch.uint8, device="cuda")
    ks = torch.full((pg.kv_rows,), 7.0, device="cuda")
    k_new, kv_new = _new_tokens(pg.rows, d, 3)
    status = _status()
    call = dsa.dsa_cache_append_q8 if q8 else dsa.dsa_cache_append
    assert call(pb, k_new, kv_new, k8, ks, kv, status) == dsa.DSA_OK
    assert int(status.item()) == dsa.DSA_DEVICE_BAD_INDEX
    written = {int(pg.phys(0, [p])[0]) for p in (297, 298, 299)}
    written |= {int(pg.phys(1, [p])[0]) for p in range(60, 64)}
    written.add(int(pg.phys(3, [0])[0]))         # the second new token of sequence 3
    changed = set(np.nonzero((kv.cpu().numpy() != 7).any(axis=1))[0].tolist())
    assert changed <= written
    assert set(np.nonzero(ks.cpu().numpy() != 7.0)[0].tolist()) == written
    assert set(np.nonzero((k8.cpu().numpy() != 7).any(axis=1))[0].tolist()) <= written


# ------------------------------------------------------------------------------- read

@pytest.mark.parametrize("d", [FULL, TINY], ids=["full", "tiny"])
@pytest.mark.parametrize("paged", [True, False])
def test_read_ranges(dsa, d, paged):
    ctx = [700, 64, 1, 130, 5000, 65]
    pg = Pages([1] * 6, ctx, paged=paged, seed=4)
    pb = pg.problem(dsa, d, 64, "decode")
    lat = ref.latents(pg.kv_rows, d, 9)
    lat[5, 3] = float("nan")
    lat[6, :128] = 2.0e38                        # a scale above 2^7 (two-step expansion)
    lat[7, :128] = 1.0e5
    packed = ref.pack_rows(lat, d)
    kv8 = torch.from_numpy(packed).cuda()
    want = torch.from_numpy(ref.unpack_rows(packed, d)).to(torch.bfloat16)
    for begin, count in ([0] * 6, ctx), ([3, 63, 0, 100, 4999, 0], [697, 1, 0, 30, 1, 65]):
        cu = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
        out = torch.full((int(cu[-1]) + 5, d["d_qk"]), 3.0, dtype=torch.bfloat16, device="cuda")
        status = _status()
        kb = None if not any(begin) else torch.tensor(begin, dtype=torch.int32, device="cuda")
        st = dsa.dsa_cache_read_q8(pb, kv8, kb, torch.from_numpy(cu).cuda(), int(cu[-1]), out,
                                   status)
        assert st == dsa.DSA_OK and int(status.item()) == 0
        rows = np.concatenate([pg.phys(b, np.arange(s, s + n))
                               for b, (s, n) in enumerate(zip(begin, count))])
        assert torch.equal(torch.nan_to_num(out[:-5].cpu().float(), nan=777.0),
                           torch.nan_to_num(want[rows].float(), nan=777.0))
        assert (out[-5:] == 3.0).all()           # rows behind the last range


def test_read_outside_the_context(dsa):
    """Keys past a context, negative keys and bad pages read as zeros and are reported; a host
    count that differs from cu_keys writes neither more nor less than both allow."""
    d = FULL
    pg = Pages([1, 1], [100, 200], seed=5)
    pb = pg.problem(dsa, d, 64, "decode")
    lat = ref.latents(pg.kv_rows, d, 10)
    packed = ref.pack_rows(lat, d)
    kv8 = torch.from_numpy(packed).cuda()
    want = torch.from_numpy(ref.unpack_rows(packed, d)).to(torch.bfloat16)
    pg.d_table[1, 1] = pg.kv_rows // 64
    cu = torch.tensor([0, 103, 303], dtype=torch.int32, device="cuda")
    kb = torch.tensor([-2, 0], dtype=torch.int32, device="cuda")
    out = torch.full((310, d["d_qk"]), 3.0, dtype=torch.bfloat16, device="cuda")
    status = _status()
    assert dsa.dsa_cache_read_q8(pb, kv8, kb, cu, 310, out, status) == dsa.DSA_OK
    assert int(status.item()) == dsa.DSA_DEVICE_BAD_INDEX
    o = out.cpu()
    assert (o[:2] == 0).all() and (o[102] == 0).all() and (o[103 + 64:103 + 128] == 0).all()
    assert torch.equal(o[2:102], want[pg.phys(0, np.arange(100))])
    assert torch.equal(o[103:167], want[pg.phys(1, np.arange(64))])
    assert torch.equal(o[231:303], want[pg.phys(1, np.arange(128, 200))])
    assert (o[303:] == 3.0).all()
    out.fill_(3.0)
    assert dsa.dsa_cache_read_q8(pb, kv8, kb, cu, 50, out, status) == dsa.DSA_OK
    assert torch.equal(out[:50].cpu()[2:], o[2:50]) and (out[50:] == 3.0).all()


# ------------------------------------------------------------------------------- attention

def _cache(pg, d, q8, seed):
    """A cache of random rows and its float64 values by physical row."""
    lat = ref.latents(pg.kv_rows, d, seed)
    if not q8:
        return lat, lat.double()
    packed = ref.pack_rows(lat, d)
    return torch.from_numpy(packed).cuda(), torch.from_numpy(ref.unpack_rows(packed, d)).cuda()


def _attend(dsa, pb, q8, q, cache, idx, rows, rb=0, rc=None, d=FULL):
    rc = rows if rc is None else rc
    out = torch.full((rows, d["h"], d["d_v"]), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, d["h"]), 9.0, device="cuda")
    size = (dsa.dsa_sparse_mla_q8_workspace_size if q8 else dsa.dsa_sparse_mla_workspace_size)
    n = size(pb, rc)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    status = _status()
    call = dsa.dsa_sparse_mla_fwd_q8 if q8 else dsa.dsa_sparse_mla_fwd
    st = call(pb, q, cache, idx, rb, rc, out, lse, ws, n, status)
    assert st == dsa.DSA_OK, dsa.status_string(st)
    torch.cuda.synchronize()
    return out, lse, int(status.item())


def _queries(rows, d, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, d["h"], d["d_qk"], generator=g, device="cuda") * scale
            ).to(torch.bfloat16)


ATT = [  # mode, new, ctx, topk
    ("decode", [1], [1], 64),
    ("decode", [1], [3000], 2048),               # few rows: split over the selection
    ("decode", [1] * 5, [1, 63, 64, 65, 700], 128),
    ("chunk", [1], [1], 64),
    ("chunk", [3, 0, 17, 1], [3, 5, 300, 4100], 2048),
    ("chunk", [64, 9], [64, 2500], 1984),        # rows from one key on; 31 tiles
    ("chunk", [90], [150], 64),                  # one tile a row
]


@pytest.mark.parametrize("mode,new,ctx,topk", ATT)
@pytest.mark.parametrize("d", [FULL, TINY], ids=["full", "tiny"])
@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
@pytest.mark.parametrize("paged", [True, False], ids=["paged", "contiguous"])
def test_attention(dsa, mode, new, ctx, topk, d, q8, paged):
    if mode == "decode" and not q8:
        pytest.skip("decode over bf16 rows is the existing operator")
    pg = Pages(new, ctx, paged=paged, seed=6)
    pb = pg.problem(dsa, d, topk, mode)
    cache, values = _cache(pg, d, q8, 21)
    q = _queries(pg.rows, d, 22)
    sigma = d["d_qk"] ** -0.5
    for holes in (0.0, 0.4):
        idx = torch.from_numpy(ref.random_selection(pg, topk, 23, holes)).cuda()
        if holes and pg.rows > 2:
            idx[1] = -1                          # a row whose mask leaves nothing
            idx[2, 64:] = -1
        out, lse, status = _attend(dsa, pb, q8, q, cache, idx, pg.rows, d=d)
        assert status == 0
        ref.check_attention_rows(out, lse, q, values, idx, pg, sigma, d, what=f"holes {holes}")


@pytest.mark.parametrize("d", [FULL, TINY], ids=["full", "tiny"])
@pytest.mark.parametrize("mode,new,ctx", [
    ("chunk", [65, 1, 0, 3], [65, 5000, 7, 2049]), ("decode", [1, 1, 1], [1, 64, 3001]),
    ("chunk", [7], [129])])
@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
def test_attention_over_every_key(dsa, d, mode, new, ctx, q8):
    """idx NULL: every prior key, of rows below and above topk."""
    if mode == "decode" and not q8:
        pytest.skip("decode over bf16 rows is the existing operator")
    pg = Pages(new, ctx, seed=7)
    pb = pg.problem(dsa, d, 2048, mode)
    cache, values = _cache(pg, d, q8, 31)
    q = _queries(pg.rows, d, 32)
    out, lse, status = _attend(dsa, pb, q8, q, cache, None, pg.rows, d=d)
    assert status == 0
    ref.check_attention_rows(out, lse, q, values, None, pg, d["d_qk"] ** -0.5, d)


@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
def test_attention_growing_logits(dsa, q8):
    """Logits that grow along the keys (up to about +-60): the running reference moves several
    times and the accumulator is rescaled."""
    d = FULL
    pg = Pages([5], [2500], seed=8)
    pb = pg.problem(dsa, d, 2048)
    lat = ref.latents(pg.kv_rows, d, 41)
    grow = torch.zeros(pg.kv_rows, device="cuda")
    grow[torch.as_tensor(pg.phys(0, np.arange(2500)), device="cuda")] = torch.linspace(
        0.05, 2.5, 2500, device="cuda")
    lat = (lat.float() * grow[:, None]).to(torch.bfloat16)
    if q8:
        packed = ref.pack_rows(lat, d)
        cache, values = torch.from_numpy(packed).cuda(), torch.from_numpy(
            ref.unpack_rows(packed, d)).cuda()
    else:
        cache, values = lat, lat.double()
    q = _queries(5, d, 42, scale=4.0)
    idx = torch.from_numpy(ref.random_selection(pg, 2048, 43)).cuda()
    out, lse, status = _attend(dsa, pb, q8, q, cache, idx, 5)
    assert status == 0
    ref.check_attention_rows(out, lse, q, values, idx, pg, d["d_qk"] ** -0.5, d)


@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
@pytest.mark.parametrize("new,ctx", [([1], [1000]), ([200], [1000])], ids=["split", "whole"])
def test_attention_one_tile(dsa, q8, new, ctx):
    """One active tile a CTA pair, at every place of the selection: 16 splits of one tile each, and
    rows whose only entries fill tile 0, 1, 2, ..."""
    d = FULL
    pg = Pages(new, ctx, seed=25)
    pb = pg.problem(dsa, d, 1024)
    cache, values = _cache(pg, d, q8, 201)
    q = _queries(pg.rows, d, 202)
    idx = torch.from_numpy(ref.random_selection(pg, 1024, 203)).cuda()
    if pg.rows > 1:
        tile = torch.arange(1024, device="cuda") // 64
        only = tile[None, :] == (torch.arange(pg.rows, device="cuda") % 12)[:, None]
        idx = torch.where(only, idx, -1)
    out, lse, status = _attend(dsa, pb, q8, q, cache, idx, pg.rows)
    assert status == 0
    ref.check_attention_rows(out, lse, q, values, idx, pg, d["d_qk"] ** -0.5, d)
    for _ in range(20):
        again, lagain, _ = _attend(dsa, pb, q8, q, cache, idx, pg.rows)
        assert torch.equal(again, out) and torch.equal(lagain, lse)


@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
@pytest.mark.parametrize("new", [[1], [160]], ids=["split", "whole"])
def test_attention_minus_infinite_logits(dsa, q8, new):
    """Selected keys whose logits are -inf (a rotary dim of -inf against a positive query) have
    probability 0, a whole first tile of them included."""
    d = FULL
    pg = Pages(new, [600], seed=26)
    pb = pg.problem(dsa, d, 256)
    lat = ref.latents(pg.kv_rows, d, 211)
    minus = np.arange(64)
    lat[torch.as_tensor(pg.phys(0, minus), device="cuda"), d["d_v"]] = float("-inf")
    if q8:
        packed = ref.pack_rows(lat, d)
        cache, values = torch.from_numpy(packed).cuda(), torch.from_numpy(
            ref.unpack_rows(packed, d)).cuda()
    else:
        cache, values = lat, lat.double()
    q = _queries(pg.rows, d, 212)
    q[:, :, d["d_v"]] = 1.0
    idx = torch.full((pg.rows, 256), -1, dtype=torch.int32, device="cuda")
    idx[:, :64] = torch.arange(64, dtype=torch.int32)
    idx[:, 64:256] = torch.arange(100, 292, dtype=torch.int32)
    rest = idx.clone()
    rest[:, :64] = -1
    out, lse, status = _attend(dsa, pb, q8, q, cache, idx, pg.rows)
    assert status == 0
    ref.check_attention_rows(out, lse, q, values, rest, pg, d["d_qk"] ** -0.5, d)


def test_rows_behind_the_last_sequence(dsa):
    """Rows that the device's cu_seqlens gives to no sequence see no keys and are reported; the
    tokens of such rows are not written."""
    d = FULL
    pg = Pages([3, 4], [70, 300], seed=27)
    pb = pg.problem(dsa, d, 128)
    cache, values = _cache(pg, d, True, 221)
    q = _queries(pg.rows, d, 222)
    idx = torch.from_numpy(ref.random_selection(pg, 128, 223)).cuda()
    out, lse, status = _attend(dsa, pb, True, q, cache, idx, pg.rows)
    assert status == 0
    pg.d_cu[2] = 5                                   # sequence 1 keeps two of its four new tokens
    pg.d_ctx[1] = 298
    o2, l2, status = _attend(dsa, pb, True, q, cache, idx, pg.rows)
    assert status == dsa.DSA_DEVICE_BAD_INDEX
    assert torch.equal(o2[:5], out[:5]) and torch.equal(l2[:5], lse[:5])
    assert (o2[5:] == 0).all() and (l2[5:] == float("-inf")).all()
    k_new, kv_new = _new_tokens(pg.rows, d, 224)
    k8 = torch.zeros(pg.kv_rows, 128, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(pg.kv_rows, device="cuda")
    before = cache.clone()
    st = _status()
    assert dsa.dsa_cache_append_q8(pb, k_new, kv_new, k8, ks, cache, st) == dsa.DSA_OK
    assert int(st.item()) == dsa.DSA_DEVICE_BAD_INDEX
    changed = (cache != before).any(dim=1).nonzero().flatten().cpu().numpy()
    places = np.concatenate([pg.phys(0, np.arange(67, 70)), pg.phys(1, np.arange(296, 298))])
    assert sorted(changed) == sorted(places)


@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
def test_attention_wide_block_table(dsa, q8):
    """A block table of more pages than are looked up in shared memory (max_seqlen past 131072)."""
    d = FULL
    pg = Pages([5, 1], [900, 70], seed=28, max_seqlen=140000)
    pb = pg.problem(dsa, d, 512)
    cache, values = _cache(pg, d, q8, 231)
    q = _queries(pg.rows, d, 232)
    idx = torch.from_numpy(ref.random_selection(pg, 512, 233, 0.2)).cuda()
    out, lse, status = _attend(dsa, pb, q8, q, cache, idx, pg.rows)
    assert status == 0
    ref.check_attention_rows(out, lse, q, values, idx, pg, d["d_qk"] ** -0.5, d)


def test_many_sequences(dsa):
    """More than 32 x 32 sequences, some without new tokens: every row finds its own."""
    d = FULL
    new = [(0, 1, 2, 1)[i % 4] for i in range(1100)]
    ctx = [n + i % 3 + (n == 0) for i, n in enumerate(new)]
    pg = Pages(new, ctx, seed=29)
    pb = pg.problem(dsa, d, 64)
    cache, values = _cache(pg, d, True, 241)
    k_new, kv_new = torch.randn(pg.rows, 128, device="cuda"), ref.latents(pg.rows, d, 242)
    k8 = torch.zeros(pg.kv_rows, 128, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(pg.kv_rows, device="cuda")
    status = _status()
    assert dsa.dsa_cache_append_q8(pb, k_new, kv_new, k8, ks, cache, status) == dsa.DSA_OK
    assert int(status.item()) == 0
    want = ref.pack_rows(kv_new, d)
    where = np.concatenate([pg.phys(*pg.row(r)).reshape(1) for r in range(pg.rows)])
    assert np.array_equal(cache.cpu().numpy()[where], want)
    values = torch.from_numpy(ref.unpack_rows(cache.cpu().numpy(), d)).cuda()
    q = _queries(pg.rows, d, 243)
    idx = torch.from_numpy(ref.random_selection(pg, 64, 244)).cuda()
    out, lse, status = _attend(dsa, pb, True, q, cache, idx, pg.rows)
    assert status == 0
    ref.check_attention_rows(out, lse, q, values, idx, pg, d["d_qk"] ** -0.5, d,
                             rows=range(0, pg.rows, 7))


@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
def test_attention_ignores_unselected_nan(dsa, q8):
    """NaN and infinities in cache rows that no entry selects (and in unused pages) change
    nothing."""
    d = FULL
    pg = Pages([6], [900], seed=9)
    pb = pg.problem(dsa, d, 512)
    lat = ref.latents(pg.kv_rows, d, 51)
    idx = torch.from_numpy(ref.random_selection(pg, 512, 52, 0.2)).cuda()
    idx[:, 200:] = -1
    used = torch.zeros(pg.kv_rows, dtype=torch.bool, device="cuda")
    used[torch.as_tensor(pg.phys(0, np.unique(idx[idx >= 0].cpu().numpy())), device="cuda")] = True
    lat[~used] = float("nan")
    if q8:
        packed = ref.pack_rows(lat, d)
        cache, values = torch.from_numpy(packed).cuda(), torch.from_numpy(
            ref.unpack_rows(packed, d)).cuda()
    else:
        cache, values = lat, lat.double()
    q = _queries(6, d, 53)
    out, lse, status = _attend(dsa, pb, q8, q, cache, idx, 6)
    assert status == 0
    ref.check_attention_rows(out, lse, q, values, idx, pg, d["d_qk"] ** -0.5, d)
    # a selected row that holds a NaN makes its query rows NaN, and only those
    first = int(pg.phys(0, [int(idx[2][idx[2] >= 0][0])])[0])
    bad = cache.clone()
    lat2 = lat[first:first + 1].clone()
    lat2[:] = float("nan")
    bad[first] = (torch.from_numpy(ref.pack_rows(lat2, d)).cuda()[0] if q8 else lat2[0])
    out2, lse2, _ = _attend(dsa, pb, q8, q, bad, idx, 6)
    hit = (idx == int(idx[2][idx[2] >= 0][0])).any(dim=1)
    assert torch.isnan(out2[hit].float()).all() and torch.equal(out2[~hit], out[~hit])
    assert torch.equal(lse2[~hit], lse[~hit])


@pytest.mark.parametrize("q8", [True, False], ids=["q8", "bf16"])
def test_attention_bad_entries(dsa, q8):
    """Indices past the row's keys, pages outside the caches, contexts that do not hold the new
    tokens: skipped and reported, the other entries and rows unaffected."""
    d = FULL
    pg = Pages([4, 3], [200, 2], seed=10, max_seqlen=256)   # sequence 1: 3 new tokens, 2 cached
    pb = pg.problem(dsa, d, 128)
    cache, values = _cache(pg, d, q8, 61)
    q = _queries(pg.rows, d, 62)
    idx = torch.full((7, 128), -1, dtype=torch.int32)
    for r in range(4):
        idx[r, :100] = torch.arange(100)
    idx[5, 0] = 0
    idx[6, :2] = torch.arange(2)
    idx = idx.cuda()
    clean, clse, status = _attend(dsa, pb, q8, q, cache, idx, 7)
    assert status == dsa.DSA_DEVICE_BAD_INDEX               # row 4 has a negative position
    ref.check_attention_rows(clean, clse, q, values, idx, pg, d["d_qk"] ** -0.5, d,
                             rows=[0, 1, 2, 3, 4, 5, 6])
    dirty = idx.clone()
    dirty[1, 100] = 198                                     # row 1 sees keys 0..197
    dirty[2, 100] = 1 << 30
    dirty[4, 0] = 0
    out, lse, status = _attend(dsa, pb, q8, q, cache, dirty, 7)
    assert status == dsa.DSA_DEVICE_BAD_INDEX
    assert torch.equal(out, clean) and torch.equal(lse, clse)
    pg.d_table[0, 1] = pg.kv_rows // 64                     # keys 64..127 of sequence 0
    out, lse, status = _attend(dsa, pb, q8, q, cache, idx, 7)
    assert status == dsa.DSA_DEVICE_BAD_INDEX
    cut = idx.clone()
    cut[:4, 64:100] = -1
    ref.check_attention_rows(out, lse, q, values, cut, pg, d["d_qk"] ** -0.5, d, rows=range(4))
    # without indices the bad page's keys are skipped the same way
    out, lse, status = _attend(dsa, pb, q8, q, cache, None, 7, rc=4)
    assert status == dsa.DSA_DEVICE_BAD_INDEX
    every = torch.full((4, 256), -1, dtype=torch.int32, device="cuda")
    for r in range(4):
        keys = [s for s in range(197 + r) if s // 64 != 1]
        every[r, :len(keys)] = torch.tensor(keys, dtype=torch.int32)
    ref.check_attention_rows(out, lse, q, values, every, pg, d["d_qk"] ** -0.5, d, rows=range(4))
    assert (out[4:] == 9.0).all() and (lse[4:] == 9.0).all()


def test_attention_row_ranges_and_noalloc(dsa):
    """A sub-range of rows writes those rows only and equals the whole call; the allocation-free
    entry point gives chunks the same result."""
    d = FULL
    pg = Pages([40, 13], [900, 3000], seed=11)
    pb = pg.problem(dsa, d, 1024)
    q = _queries(pg.rows, d, 72)
    idx = torch.from_numpy(ref.random_selection(pg, 1024, 73)).cuda()
    for q8 in (True, False):
        cache, values = _cache(pg, d, q8, 71)
        whole, wl, _ = _attend(dsa, pb, q8, q, cache, idx, pg.rows)
        for rb, rc in ((0, 1), (7, 40), (52, 1), (10, 0)):
            out, lse, status = _attend(dsa, pb, q8, q, cache, idx[rb:rb + rc].contiguous(), pg.rows,
                                       rb, rc)
            assert status == 0
            ref.check_attention_rows(out, lse, q, values, idx, pg, d["d_qk"] ** -0.5, d,
                                     rows=range(rb, rb + rc))
            keep = [r for r in range(pg.rows) if not rb <= r < rb + rc]
            assert (out[keep] == 9.0).all() and (lse[keep] == 9.0).all()
    out, lse = torch.empty_like(whole), torch.empty_like(wl)
    for rc in (2, 53):
        assert dsa.dsa_sparse_mla_fwd_noalloc(pb, q, cache, idx, 0, rc, out, lse) == dsa.DSA_OK
        torch.cuda.synchronize()
        ref.check_attention_rows(out, lse, q, values, idx, pg, d["d_qk"] ** -0.5, d,
                                 rows=range(rc))


def test_cache_past_32_bits(dsa):
    """Rows whose byte offset passes 2^32: written, read back and attended."""
    d = FULL
    rows = (1 << 32) // 656 + 70000
    rows = (rows + 63) // 64 * 64
    pg = Pages([5, 1], [150, 700], seed=12)
    pg.table = pg.table + (rows - pg.kv_rows) // 64          # every page at the far end
    pg.d_table = torch.from_numpy(pg.table).cuda()
    pg.kv_rows = rows
    pb = pg.problem(dsa, d, 256)
    kv8 = torch.zeros(rows, 656, dtype=torch.uint8, device="cuda")
    k8 = torch.zeros(rows, 128, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(rows, device="cuda")
    all_pg = Pages([150, 700], [150, 700], seed=12)
    all_pg.table, all_pg.d_table, all_pg.kv_rows = pg.table, pg.d_table, rows
    apb = all_pg.problem(dsa, d, 256)
    k_new, kv_new = _new_tokens(850, d, 81)
    kv_new = ref.latents(850, d, 82)
    status = _status()
    assert dsa.dsa_cache_append_q8(apb, k_new, kv_new, k8, ks, kv8, status) == dsa.DSA_OK
    packed = ref.pack_rows(kv_new, d)
    phys = torch.from_numpy(np.concatenate([all_pg.phys(0, np.arange(150)),
                                            all_pg.phys(1, np.arange(700))])).cuda()
    assert np.array_equal(kv8[phys].cpu().numpy(), packed)
    back = torch.empty(850, 576, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 150, 850], dtype=torch.int32, device="cuda")
    assert dsa.dsa_cache_read_q8(apb, kv8, None, cu, 850, back, status) == dsa.DSA_OK
    val = torch.from_numpy(ref.unpack_rows(packed, d)).cuda()
    assert torch.equal(back.double(), val)
    near = Pages([5, 1], [150, 700], paged=False)            # the values in logical order
    near.phys = lambda b, pos: np.asarray(pos, np.int64) + (0, 150)[b]
    q = _queries(6, d, 83)
    idx = torch.from_numpy(ref.random_selection(pg, 256, 84)).cuda()
    out, lse, st = _attend(dsa, pb, True, q, kv8, idx, 6)
    assert st == 0 and int(status.item()) == 0
    ref.check_attention_rows(out, lse, q, val, idx, near, d["d_qk"] ** -0.5, d)


# ------------------------------------------------------------------------------- selection

@pytest.mark.parametrize("d", [FULL, TINY], ids=["full", "tiny"])
@pytest.mark.parametrize("layout", ["paged", "contiguous", "interleaved"])
@pytest.mark.parametrize("new,ctx", [
    ([1], [1]), ([5, 0, 64, 1, 2, 130], [5, 77, 130, 1000, 333, 2049]),
    ([4] * 40, [100 + 61 * i for i in range(40)])])
def test_chunk_scores_and_topk(dsa, d, layout, new, ctx):
    """Scores within the indexer's tolerance, nothing written past a row's position, and the
    top-k exact on them, with and without the indexer's counts and over row sub-ranges."""
    pg = Pages(new, ctx, paged=layout != "contiguous", seed=13)
    topk = 64
    pb = pg.problem(dsa, d, topk)
    q8, qs, w, k8, ks = ref.indexer_inputs(pg.rows, pg.kv_rows, d, 91)
    kin, sin = (ref.interleave(k8, ks), None) if layout == "interleaved" else (k8, ks)
    ld = (max(ctx) + 3) // 4 * 4
    full = d is FULL
    for rb, rc in ((0, pg.rows), (pg.rows // 3, pg.rows - pg.rows // 2)):
        slab = torch.full((rc, ld), -7.0, device="cuda")
        hist = torch.zeros(rc, 2048, dtype=torch.int32, device="cuda") if full else None
        status = _status()
        assert dsa.dsa_indexer_scores(pb, q8, qs, w, kin, sin, rb, rc, slab, ld, status,
                                      hist=hist) == dsa.DSA_OK
        assert int(status.item()) == 0
        got = to_np(slab)
        rows = range(rc) if rc < 60 else list(range(0, rc, 7)) + [rc - 1]
        for i in rows:
            want = ref.scores_row(q8, qs, w, k8, ks, pg, rb + i).cpu().numpy()
            check_scores(got[i, :len(want)], want, f"row {rb + i}")
        for i in range(rc):
            _, pos = pg.row(rb + i)
            assert (got[i, pos + 1:] == -7.0).all()
            if full:
                assert int(hist[i].sum()) == pos + 1
        idx = torch.empty(rc, topk, dtype=torch.int32, device="cuda")
        assert dsa.dsa_topk(pb, slab, ld, rb, rc, idx, status) == dsa.DSA_OK
        for i in rows:
            _, pos = pg.row(rb + i)
            check_topk_exact(to_np(idx)[i], got[i, :pos + 1], topk, f"row {rb + i}")
        if full:
            idx2 = torch.empty_like(idx)
            assert dsa.dsa_topk(pb, slab, ld, rb, rc, idx2, status, hist=hist) == dsa.DSA_OK
            assert torch.equal(idx, idx2) and not hist.any()
        n = dsa.dsa_indexer_topk_workspace_size(pb, rc)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        idx3 = torch.empty_like(idx)
        sel = torch.empty(rc, topk, device="cuda")
        assert dsa.dsa_indexer_topk(pb, q8, qs, w, kin, sin, rb, rc, idx3, ws, n, status,
                                    sel_out=sel) == dsa.DSA_OK
        assert torch.equal(idx, idx3) and int(status.item()) == 0
        pick = torch.gather(slab, 1, idx.clamp_min(0).long())
        assert torch.equal(sel, torch.where(idx >= 0, pick, 0.0))


def test_chunk_scores_bad_geometry(dsa):
    """A page outside the caches and a context shorter than its new tokens are reported; rows
    without keys select nothing."""
    d = FULL
    pg = Pages([4, 3], [200, 2], seed=14, max_seqlen=256)
    pb = pg.problem(dsa, d, 64)
    q8, qs, w, k8, ks = ref.indexer_inputs(7, pg.kv_rows, d, 95)
    slab = torch.full((7, 256), -7.0, device="cuda")
    status = _status()
    assert dsa.dsa_indexer_scores(pb, q8, qs, w, k8, ks, 0, 7, slab, 256, status) == dsa.DSA_OK
    assert int(status.item()) == dsa.DSA_DEVICE_BAD_INDEX
    for r in (0, 3, 5, 6):
        want = ref.scores_row(q8, qs, w, k8, ks, pg, r).cpu().numpy()
        check_scores(to_np(slab)[r, :len(want)], want, f"row {r}")
    assert (slab[4] == -7.0).all()
    idx = torch.empty(7, 64, dtype=torch.int32, device="cuda")
    assert dsa.dsa_topk(pb, slab, 256, 0, 7, idx, status) == dsa.DSA_OK
    assert (idx[4] == -1).all() and idx[5, 0] == 0 and (idx[5, 1:] == -1).all()
    status.zero_()
    pg.d_ctx[1] = 3
    pg.d_table[0, 1] = -5
    assert dsa.dsa_indexer_scores(pb, q8, qs, w, k8, ks, 0, 7, slab, 256, status) == dsa.DSA_OK
    assert int(status.item()) == dsa.DSA_DEVICE_BAD_INDEX
    want = ref.scores_row(q8, qs, w, k8, ks, pg, 2).cpu().numpy()
    keep = np.r_[0:64, 128:len(want)]
    check_scores(to_np(slab)[2, keep], want[keep], "other pages")


# ------------------------------------------------------------------------------- whole path

def _step(dsa, pg, d, topk, q8, mode, seed):
    """Append, select and attend one step through the public calls; returns everything."""
    pb = pg.problem(dsa, d, topk, mode)
    k_new, kv_new = _new_tokens(pg.rows, d, seed)
    kv_new = ref.latents(pg.rows, d, seed + 1)
    qi, qs, w, k8, ks = ref.indexer_inputs(pg.rows, pg.kv_rows, d, seed + 2)
    lat = ref.latents(pg.kv_rows, d, seed + 3)
    cache = torch.from_numpy(ref.pack_rows(lat, d)).cuda() if q8 else lat
    q = _queries(pg.rows, d, seed + 4)
    status = _status()
    append = dsa.dsa_cache_append_q8 if q8 else dsa.dsa_cache_append
    assert append(pb, k_new, kv_new, k8, ks, cache, status) == dsa.DSA_OK
    size = dsa.dsa_forward_q8_workspace_size if q8 else dsa.dsa_forward_workspace_size
    n = size(pb)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    idx = torch.empty(pg.rows, topk, dtype=torch.int32, device="cuda")
    sel = torch.empty(pg.rows, topk, device="cuda")
    out = torch.empty(pg.rows, d["h"], d["d_v"], dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(pg.rows, d["h"], device="cuda")
    forward = dsa.dsa_forward_q8 if q8 else dsa.dsa_forward
    run = lambda i, s: forward(pb, qi, qs, w, k8, ks, q, cache, i, out, lse, ws, n, status,
                               sel_out=s)
    assert run(idx, sel) == dsa.DSA_OK
    assert int(status.item()) == 0
    values = (torch.from_numpy(ref.unpack_rows(cache.cpu().numpy(), d)).cuda() if q8
              else cache.double())
    return dict(pb=pb, qi=qi, qs=qs, w=w, k8=k8, ks=ks, q=q, cache=cache, values=values, idx=idx,
                sel=sel, out=out, lse=lse, ws=ws, n=n, status=status, run=run)


@pytest.mark.parametrize("q8,mode,new,ctx,topk", [
    (True, "chunk", [70, 1, 4, 0, 33], [70, 5000, 2100, 9, 2500], 2048),
    (False, "chunk", [70, 1, 4, 0, 33], [70, 5000, 2100, 9, 2500], 2048),
    (True, "decode", [1] * 6, [1, 64, 2049, 2048, 4000, 3333], 2048),
    (True, "chunk", [20, 3], [150, 64], 192),
])
def test_forward(dsa, q8, mode, new, ctx, topk):
    d = FULL
    pg = Pages(new, ctx, seed=15)
    s = _step(dsa, pg, d, topk, q8, mode, 101)
    ld = (max(ctx) + 3) // 4 * 4
    slab = torch.zeros(pg.rows, ld, device="cuda")
    assert dsa.dsa_indexer_scores(s["pb"], s["qi"], s["qs"], s["w"], s["k8"], s["ks"], 0, pg.rows,
                                  slab, ld, s["status"]) == dsa.DSA_OK
    got = to_np(slab)
    for r in range(pg.rows):
        _, pos = pg.row(r)
        want = ref.scores_row(s["qi"], s["qs"], s["w"], s["k8"], s["ks"], pg, r).cpu().numpy()
        check_scores(got[r, :pos + 1], want, f"row {r}")
        check_topk_exact(to_np(s["idx"])[r], got[r, :pos + 1], topk, f"row {r}")
    ref.check_attention_rows(s["out"], s["lse"], s["q"], s["values"], s["idx"], pg,
                             d["d_qk"] ** -0.5, d)
    # without the indices: the same selection, attended the same way
    out, lse = s["out"].clone(), s["lse"].clone()
    s["out"].fill_(9.0)
    assert s["run"](None, None) == dsa.DSA_OK
    torch.cuda.synchronize()
    assert torch.equal(s["out"], out) and torch.equal(s["lse"], lse)


def test_forward_short_contexts_skip_the_indexer(dsa):
    """No context above topk and no indices kept: every key is attended."""
    pg = Pages([9, 2], [120, 64], seed=16)
    for q8 in (True, False):
        s = _step(dsa, pg, FULL, 128, q8, "chunk", 111)
        assert s["run"](None, None) == dsa.DSA_OK
        torch.cuda.synchronize()
        ref.check_attention_rows(s["out"], s["lse"], s["q"], s["values"], None, pg, 576 ** -0.5,
                                 FULL)


def test_forward_in_several_launches(dsa):
    """A chunk whose scores pass the slab budget runs in several launches of whole rows: the same
    indices and outputs as row by row through the stage calls; and row ranges match."""
    d = FULL
    pg = Pages([900, 30], [90000, 131072], seed=17)
    assert dsa.dsa_forward_chunk_rows_for(pg.problem(dsa, d, 2048), 0, 148) < pg.rows
    s = _step(dsa, pg, d, 2048, True, "chunk", 121)
    rows = [0, 1, 443, 444, 445, 887, 888, 899, 900, 929]
    for r in rows:
        want = ref.scores_row(s["qi"], s["qs"], s["w"], s["k8"], s["ks"], pg, r).cpu().numpy()
        got = to_np(s["idx"])[r]
        _, pos = pg.row(r)
        valid = got[got >= 0]
        assert len(valid) == 2048 and (np.diff(valid) > 0).all() and valid.max() <= pos
        sel = to_np(s["sel"])[r]
        check_scores(sel, want[valid], f"row {r}")
        cut = np.sort(want)[-2048]
        tol = 1e-3 * abs(cut) + 1e-5 * want.max()
        assert (want[valid] >= cut - tol).all()
    ref.check_attention_rows(s["out"], s["lse"], s["q"], s["values"], s["idx"], pg, 576 ** -0.5, d,
                             rows=rows)


def test_forward_rows_of_a_chunk(dsa):
    """dsa_forward_rows on a chunk problem: query-side arrays of the range only."""
    d = FULL
    pg = Pages([50, 7], [2600, 400], seed=18)
    s = _step(dsa, pg, d, 2048, False, "chunk", 131)
    for rb, rc in ((3, 30), (44, 13)):
        part = slice(rb, rb + rc)
        cut = lambda t: t[part].clone()
        idx = torch.empty(rc, 2048, dtype=torch.int32, device="cuda")
        out = torch.empty(rc, 128, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(rc, 128, device="cuda")
        st = dsa.dsa_forward_rows(s["pb"], rb, rc, cut(s["qi"]), cut(s["qs"]), cut(s["w"]), s["k8"],
                                  s["ks"], cut(s["q"]), s["cache"], idx, out, lse, s["ws"], s["n"],
                                  s["status"])
        assert st == dsa.DSA_OK and int(s["status"].item()) == 0
        assert torch.equal(idx, s["idx"][part])
        shift = type("P", (), {"row": lambda self, r: pg.row(r + rb), "rows": rc,
                               "phys": lambda self, b, p: pg.phys(b, p)})()
        ref.check_attention_rows(out, lse, cut(s["q"]), s["values"], idx, shift, 576 ** -0.5, d)


def test_chunk_of_single_tokens_equals_decode(dsa):
    """One new token per sequence is the same problem in both modes: the same rows written, the
    same scores and selection, attention within its bound."""
    d = FULL
    pg = Pages([1] * 7, [1, 65, 4000, 2048, 2049, 700, 3001], seed=19)
    a = _step(dsa, pg, d, 2048, True, "chunk", 141)
    b = _step(dsa, pg, d, 2048, True, "decode", 141)
    assert torch.equal(a["cache"], b["cache"]) and torch.equal(a["k8"], b["k8"])
    assert torch.equal(a["idx"], b["idx"]) and torch.equal(a["out"], b["out"])
    assert torch.equal(a["lse"], b["lse"])


def test_captured_step_replays(dsa):
    """A step (append, forward, read back) captured into a CUDA graph and replayed with other
    inputs, contexts and pages in the same buffers equals the eager calls, on another stream."""
    d, topk = FULL, 2048
    pg = Pages([1, 4, 20], [2500, 700, 3000], seed=20)
    pb = pg.problem(dsa, d, topk)
    names = dict(k_new=(pg.rows, 128), kv_new=(pg.rows, 576), q=(pg.rows, 128, 576))
    qi, qs, w, k8, ks = ref.indexer_inputs(pg.rows, pg.kv_rows, d, 151)
    k_new = torch.zeros(names["k_new"], device="cuda")
    kv_new = torch.zeros(names["kv_new"], dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(names["q"], dtype=torch.bfloat16, device="cuda")
    kv8 = torch.from_numpy(ref.pack_rows(ref.latents(pg.kv_rows, d, 152), d)).cuda()
    n = dsa.dsa_forward_q8_workspace_size(pb)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    status = _status()
    cu = torch.tensor([0, 2500, 3200, 6200], dtype=torch.int32, device="cuda")

    def outputs():
        return (torch.zeros(pg.rows, topk, dtype=torch.int32, device="cuda"),
                torch.zeros(pg.rows, 128, 512, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(pg.rows, 128, device="cuda"),
                torch.zeros(6200, 576, dtype=torch.bfloat16, device="cuda"))

    def step(o):
        dsa.check(dsa.dsa_cache_append_q8(pb, k_new, kv_new, k8, ks, kv8, status))
        dsa.check(dsa.dsa_forward_q8(pb, qi, qs, w, k8, ks, q, kv8, o[0], o[1], o[2], ws, n,
                                     status))
        dsa.check(dsa.dsa_cache_read_q8(pb, kv8, None, cu, 6200, o[3], status))

    graph_out, eager_out = outputs(), outputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(graph_out)                              # warm-up before the capture
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(graph_out)
    for trial in range(3):
        g = torch.Generator(device="cuda").manual_seed(160 + trial)
        k_new.normal_(generator=g)
        kv_new.copy_(ref.latents(pg.rows, d, 170 + trial))
        q.copy_(_queries(pg.rows, d, 180 + trial))
        pg.d_ctx.copy_(torch.tensor([[2500, 700, 3000], [1, 699, 20], [2049, 4, 2999]][trial],
                                    dtype=torch.int32))
        status.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        status.zero_()                               # (the read asks for more than the contexts)
        step(eager_out)
        torch.cuda.synchronize()
        for a, b in zip(graph_out, eager_out):
            assert torch.equal(a, b)


def test_two_streams_at_once(dsa):
    """Two calls in flight on two streams with their own workspaces do not disturb each other."""
    d = FULL
    pg = Pages([1, 3], [3000, 2800], seed=21)
    pb = pg.problem(dsa, d, 2048)
    cache, _ = _cache(pg, d, True, 191)
    idx = torch.from_numpy(ref.random_selection(pg, 2048, 192)).cuda()
    n = dsa.dsa_sparse_mla_q8_workspace_size(pb, pg.rows)
    qs = [_queries(pg.rows, d, 193 + i) for i in range(2)]
    want = [_attend(dsa, pb, True, q, cache, idx, pg.rows) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty_like(want[0][0]), torch.empty_like(want[0][1]),
             torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, s, (o, l, ws) in zip(qs, streams, outs):
            assert dsa.dsa_sparse_mla_fwd_q8(pb, q, cache, idx, 0, pg.rows, o, l, ws, n,
                                             stream=s) == dsa.DSA_OK
    torch.cuda.synchronize()
    for (o, l, _), (wo, wl, _) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)


def test_workspace_too_small(dsa):
    d = FULL
    pg = Pages([1], [3000], seed=22)
    pb = pg.problem(dsa, d, 2048)
    n = dsa.dsa_sparse_mla_q8_workspace_size(pb, 1)
    assert n > 0                                     # one long row is split
    t = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    assert dsa.dsa_sparse_mla_fwd_q8(pb, t, t, t, 0, 1, t, t, t, n - 1) == \
        dsa.DSA_ERR_WORKSPACE_TOO_SMALL
    m = dsa.dsa_forward_q8_workspace_size(pb)
    assert dsa.dsa_forward_q8(pb, t, t, t, t, t, t, t, None, t, t, t, m - 1) == \
        dsa.DSA_ERR_WORKSPACE_TOO_SMALL
    # every prior key of contexts past 131072 is refused
    far = dsa.make_problem(mode="chunk", topk=2048, softmax_scale=0.04, num_kv_rows=1 << 30,
                           seqlens=[4000], cu_seqlens=pg.d_cu, seq_lens=pg.d_ctx, block_table=None,
                           max_seqlen=131073, **d)
    assert dsa.dsa_sparse_mla_fwd_q8(far, t, t, None, 0, 4000, t, t, t, 1 << 40) == \
        dsa.DSA_ERR_UNSUPPORTED_SHAPE
