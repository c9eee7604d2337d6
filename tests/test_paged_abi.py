"""Argument checks of the chunk mode and the 8-bit latent cache, refused before any launch, and
the 64-bit definitions their GPU tests compare with, pinned on the CPU."""
import numpy as np
import pytest
import torch

from tests import paged_ref as ref
from tests.test_abi import FAKE, dsa  # noqa: F401  (the fixture that builds the library)

FULL = dict(h_idx=64, d_idx=128, h=128, d_qk=576, d_v=512, topk=2048, softmax_scale=0.04)


def _chunk(dsa, new=(5, 0, 100), max_seqlen=4096, kv_rows=1 << 20, table=FAKE, **kw):  # noqa: F811
    args = dict(FULL, **kw)
    pb = dsa.make_problem(mode="chunk", num_kv_rows=kv_rows, seqlens=list(new), cu_seqlens=FAKE,
                          max_seqlen=max_seqlen, **args)
    pb.seqs.seq_lens = FAKE
    pb.seqs.block_table = table
    pb.seqs.max_blocks = 64
    return pb


def _decode(dsa, batch=2, **kw):  # noqa: F811
    pb = dsa.make_problem(mode="decode", num_kv_rows=1 << 20, seqlens=[4096] * batch,
                          max_seqlen=4096, **dict(FULL, **kw))
    pb.seqs.seq_lens = FAKE
    return pb


def _prefill(dsa):  # noqa: F811
    return dsa.make_problem(mode="prefill", num_kv_rows=1 << 20, seqlens=[100], cu_seqlens=FAKE,
                            **FULL)


def test_make_problem_modes(dsa):  # noqa: F811
    pb = _chunk(dsa)
    assert pb.seqs.mode == dsa.DSA_CHUNK == 2 and pb.seqs.total_rows == 105
    with pytest.raises(ValueError):
        dsa.make_problem(mode="chunk", num_kv_rows=64, seqlens=[1], cu_seqlens=FAKE, **FULL)
    with pytest.raises(ValueError):
        dsa.make_problem(mode="extend", num_kv_rows=64, seqlens=[1], max_seqlen=1, **FULL)


def test_chunk_geometry_refused(dsa):  # noqa: F811
    f5 = [FAKE] * 5
    scores = lambda pb: dsa.dsa_indexer_scores(pb, *f5, 0, 1, FAKE, 4096, None, 0)
    pb = _chunk(dsa)
    pb.seqs.mode = 3
    assert scores(pb) == dsa.DSA_ERR_INVALID_ARG
    for field in ("seq_lens", "cu_seqlens", "cu_seqlens_host"):
        pb = _chunk(dsa)
        setattr(pb.seqs, field, None)
        assert scores(pb) == dsa.DSA_ERR_INVALID_ARG, field
    pb = _chunk(dsa)
    pb.seqs.total_rows = 104                                  # not cu_seqlens[batch]
    assert scores(pb) == dsa.DSA_ERR_INVALID_ARG
    assert scores(_chunk(dsa, new=(5000,))) == dsa.DSA_ERR_INVALID_ARG      # above max_seqlen
    pb = _chunk(dsa)
    pb.seqs.max_blocks = 63
    assert scores(pb) == dsa.DSA_ERR_INVALID_ARG
    assert scores(_chunk(dsa, table=None, kv_rows=4096)) == dsa.DSA_ERR_INVALID_ARG
    assert scores(_chunk(dsa, block_size=32)) == dsa.DSA_ERR_UNSUPPORTED_SHAPE
    # the slab must hold the longest context, whatever the rows
    assert dsa.dsa_topk(_chunk(dsa), FAKE, 4092, 0, 1, FAKE, None, 0) == dsa.DSA_ERR_INVALID_ARG
    assert dsa.dsa_topk(_chunk(dsa), FAKE, 4096, 100, 6, FAKE, None, 0) == dsa.DSA_ERR_INVALID_ARG
    # scales inside the key pages need pages
    assert dsa.dsa_indexer_scores(_chunk(dsa, table=None), FAKE, FAKE, FAKE, FAKE, None, 0, 1, FAKE,
                                  4096, None, 0) == dsa.DSA_ERR_INVALID_ARG


def test_training_refuses_chunks(dsa):  # noqa: F811
    pb = _chunk(dsa, max_seqlen=2048)
    f = [FAKE] * 4
    inv = dsa.DSA_ERR_INVALID_ARG
    assert dsa.dsa_indexer_kl_target(pb, *f, 0, 1, FAKE, None, 0) == inv
    assert dsa.dsa_indexer_kl_target_dense(pb, FAKE, FAKE, FAKE, 0, 1, FAKE, 2048, None, 0) == inv
    assert dsa.dsa_indexer_kl_backward(pb, *[FAKE] * 7, 0, 1, *f, None, 0) == inv
    assert dsa.dsa_indexer_kl_backward_dense(pb, *[FAKE] * 6, 2048, 0, 1, *f, None, 0) == inv


def test_append_q8_refusals(dsa):  # noqa: F811
    call = lambda p, a: dsa.dsa_cache_append_q8(p, *a, None, 0)
    ok = [FAKE] * 5
    for pb in (_chunk(dsa), _decode(dsa)):
        for i in (0, 1, 2, 4):
            assert call(pb, ok[:i] + [None] + ok[i + 1:]) == dsa.DSA_ERR_INVALID_ARG, i
        for i in range(5):
            assert call(pb, ok[:i] + [FAKE + 8] + ok[i + 1:]) == dsa.DSA_ERR_MISALIGNED, i
    assert call(_decode(dsa), ok[:3] + [None] + ok[4:]) == dsa.DSA_ERR_INVALID_ARG  # no pages
    assert call(_prefill(dsa), ok) == dsa.DSA_ERR_INVALID_ARG
    assert call(_chunk(dsa, d_qk=512), ok) == dsa.DSA_ERR_UNSUPPORTED_SHAPE
    assert call(_chunk(dsa, d_idx=32), ok) == dsa.DSA_ERR_UNSUPPORTED_SHAPE
    assert call(_chunk(dsa, new=(0, 0)), ok) == dsa.DSA_OK               # no new tokens


def test_read_q8_refusals(dsa):  # noqa: F811
    def call(p, kv8=FAKE, kb=None, cu=FAKE, n=5, out=FAKE):
        return dsa.dsa_cache_read_q8(p, kv8, kb, cu, n, out, None, 0)
    pb = _decode(dsa)
    for kw in (dict(kv8=None), dict(cu=None), dict(out=None), dict(n=-1)):
        assert call(pb, **kw) == dsa.DSA_ERR_INVALID_ARG, kw
    for kw in (dict(kv8=FAKE + 4), dict(kb=FAKE + 4), dict(cu=FAKE + 4), dict(out=FAKE + 2)):
        assert call(pb, **kw) == dsa.DSA_ERR_MISALIGNED, kw
    assert call(_prefill(dsa)) == dsa.DSA_ERR_INVALID_ARG
    assert call(_decode(dsa, d_v=576)) == dsa.DSA_ERR_UNSUPPORTED_SHAPE
    assert call(pb, n=0) == dsa.DSA_OK


def test_attention_q8_refusals(dsa):  # noqa: F811
    def call(p, q=FAKE, kv8=FAKE, idx=FAKE, rb=0, rc=1, out=FAKE, lse=FAKE, ws=None):
        return dsa.dsa_sparse_mla_fwd_q8(p, q, kv8, idx, rb, rc, out, lse, ws, 0, None, 0)
    pb = _chunk(dsa)
    for kw in (dict(q=None), dict(kv8=None), dict(out=None), dict(lse=None), dict(rb=-1),
               dict(rb=105), dict(rc=106)):
        assert call(pb, **kw) == dsa.DSA_ERR_INVALID_ARG, kw
    for kw in (dict(q=FAKE + 8), dict(kv8=FAKE + 8), dict(idx=FAKE + 4), dict(out=FAKE + 2),
               dict(lse=FAKE + 4), dict(ws=FAKE + 8)):
        assert call(pb, **kw) == dsa.DSA_ERR_MISALIGNED, kw
    assert call(_prefill(dsa)) == dsa.DSA_ERR_INVALID_ARG
    assert call(_chunk(dsa, h=64)) == dsa.DSA_ERR_UNSUPPORTED_SHAPE
    assert dsa.dsa_forward_q8(_prefill(dsa), *[FAKE] * 7, None, FAKE, FAKE, FAKE, 1 << 40, None,
                              0) == dsa.DSA_ERR_INVALID_ARG
    assert dsa.dsa_forward_q8(pb, *[FAKE] * 6, None, None, FAKE, FAKE, FAKE, 1 << 40, None,
                              0) == dsa.DSA_ERR_INVALID_ARG
    # scores are kept only with the indices
    assert dsa.dsa_forward_q8(pb, *[FAKE] * 7, None, FAKE, FAKE, FAKE, 1 << 40, None, 0,
                              sel_out=FAKE) == dsa.DSA_ERR_INVALID_ARG


def test_row_bytes_and_plans(dsa):  # noqa: F811
    tiny = dict(h_idx=4, d_idx=32, h=16, d_qk=160, d_v=128, topk=64)
    assert dsa.dsa_q8_row_bytes(_decode(dsa)) == ref.row_bytes(ref.FULL) == 656
    assert dsa.dsa_q8_row_bytes(_decode(dsa, **tiny)) == ref.row_bytes(ref.TINY) == 208
    assert dsa.dsa_q8_row_bytes(_decode(dsa, d_qk=512)) == 0
    # 128k contexts: 512 rows of scores per 256 MiB, cut to whole waves of 74 two-CTA rows
    pb = _chunk(dsa, new=(2000,), max_seqlen=131072, kv_rows=1 << 20)
    pb.seqs.max_blocks = 2048
    assert dsa.dsa_forward_chunk_rows_for(pb, 0, 148) == 444
    assert dsa.dsa_forward_chunk_rows_for(_chunk(dsa), 0, 148) == 105
    size = dsa.dsa_forward_workspace_size_for(pb, 148)
    assert size >= 444 * 131072 * 4 + 444 * 2048 * 4 + 444 * 2048 * 4
    assert dsa.dsa_forward_workspace_size_for(_chunk(dsa, new=(0,)), 148) == 0


def test_definitions_against_torch_casts():
    """The 64-bit packing against torch's e4m3 cast and its error bound, on ordinary, extreme and
    tie values."""
    g = torch.Generator().manual_seed(3)
    d = ref.FULL
    x = (torch.randn(64, d["d_qk"], generator=g) *
         torch.exp(4 * torch.randn(64, 1, generator=g))).to(torch.bfloat16)
    x[0] = 0
    x[1, :128] = torch.tensor(3.0e38)
    x[2, :128] = torch.tensor(1.0e-38)
    x[3, :128] = torch.linspace(-1, 1, 128).to(torch.bfloat16) * 448
    rows = ref.pack_rows(x, d)
    assert rows.shape == (64, 656)
    scale = np.ascontiguousarray(rows[:, 512:528]).view(np.float32)
    assert (np.frexp(scale)[0] == 0.5).all()                          # powers of two
    val = x[:, :512].double().numpy().reshape(64, 4, 128)
    top = np.abs(val).max(axis=2)
    mid = (top > 0) & (scale > 2.0 ** -100) & (scale < 2.0 ** 119)
    assert (top[mid] <= 448 * scale[mid]).all() and (top[mid] > 224 * scale[mid]).all()
    y = torch.from_numpy(val / scale[:, :, None].astype(np.float64)).clamp(-448, 448)
    cast = y.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(64, 512)
    assert np.array_equal(cast, rows[:, :512])
    back = ref.unpack_rows(rows, d)
    err = np.abs(back[:, :512] - x[:, :512].double().numpy()).reshape(64, 4, 128)
    bound = 2.0 ** -4 * np.abs(val) + 2.0 ** -10 * scale[:, :, None]
    assert (err <= bound)[mid].all()
    assert np.array_equal(back[:, 512:], x[:, 512:].double().numpy())
    # what is read back is exact in bf16
    b16 = torch.from_numpy(back).to(torch.bfloat16).double().numpy()
    assert np.array_equal(b16, back)
    x[5, 130] = float("inf")
    x[6, 300] = float("nan")
    back = ref.unpack_rows(ref.pack_rows(x, d), d)
    assert np.isnan(back[5, 128:256]).all() and np.isfinite(back[5, :128]).all()
    assert np.isnan(back[6, 256:384]).all() and np.isfinite(back[6, 384:]).all()
