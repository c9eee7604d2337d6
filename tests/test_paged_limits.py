"""Limits of attention over the paged caches: 131072 keys a context without indices, whatever the rows,
and positive softmax scales (checked before any device is touched, with addresses that are never
read)."""
import pytest

from tests.test_abi import FAKE, dsa  # noqa: F401  (the fixture that builds the library)
from tests.test_paged_abi import FULL

LIMIT = 131072


def _pb(dsa, mode, rows, max_seqlen):  # noqa: F811
    new = [1] * rows if mode == "decode" else [rows]
    pb = dsa.make_problem(mode=mode, num_kv_rows=1 << 30, seqlens=new, cu_seqlens=FAKE,
                          max_seqlen=max_seqlen, **FULL)
    pb.seqs.seq_lens = FAKE
    pb.seqs.block_table = FAKE
    pb.seqs.max_blocks = (max_seqlen + 63) // 64
    return pb


@pytest.mark.parametrize("rows", [1, 4, 4000])
def test_every_key_of_a_context_past_the_limit_is_refused(dsa, rows):  # noqa: F811
    for mode in ("decode", "chunk"):
        pb = _pb(dsa, mode, rows, LIMIT + 1)
        assert dsa.dsa_sparse_mla_fwd_q8(pb, FAKE, FAKE, None, 0, rows, FAKE, FAKE, FAKE, 1 << 40,
                                         None, 0) == dsa.DSA_ERR_UNSUPPORTED_SHAPE
    pb = _pb(dsa, "chunk", rows, LIMIT + 1)
    assert dsa.dsa_sparse_mla_fwd(pb, FAKE, FAKE, None, 0, rows, FAKE, FAKE, FAKE, 1 << 40, None,
                                  0) == dsa.DSA_ERR_UNSUPPORTED_SHAPE
    assert dsa.dsa_sparse_mla_fwd_noalloc(pb, FAKE, FAKE, None, 0, rows, FAKE, FAKE, None,
                                          0) == dsa.DSA_ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("sigma", [0.0, -0.04, float("inf"), float("nan")])
def test_softmax_scales_that_are_not_positive_are_refused(dsa, sigma):  # noqa: F811
    """A mask of -inf times such a scale is no mask."""
    inv = dsa.DSA_ERR_INVALID_ARG
    f = [FAKE] * 7
    for mode in ("decode", "chunk"):
        pb = _pb(dsa, mode, 2, 4096)
        pb.dims.softmax_scale = sigma
        assert dsa.dsa_sparse_mla_fwd_q8(pb, FAKE, FAKE, FAKE, 0, 2, FAKE, FAKE, FAKE, 1 << 40,
                                         None, 0) == inv
        assert dsa.dsa_forward_q8(pb, *f, None, FAKE, FAKE, FAKE, 1 << 40, None, 0) == inv
    pb = _pb(dsa, "chunk", 2, 4096)
    pb.dims.softmax_scale = sigma
    assert dsa.dsa_sparse_mla_fwd(pb, FAKE, FAKE, FAKE, 0, 2, FAKE, FAKE, FAKE, 1 << 40, None,
                                  0) == inv
    assert dsa.dsa_sparse_mla_fwd_noalloc(pb, FAKE, FAKE, FAKE, 0, 2, FAKE, FAKE, None, 0) == inv
    assert dsa.dsa_forward(pb, *f, None, FAKE, FAKE, FAKE, 1 << 40, None, 0) == inv
    assert dsa.dsa_forward_rows(pb, 0, 1, *f, None, FAKE, FAKE, FAKE, 1 << 40, None, 0) == inv
    # the calls that do not attend take any scale (here: past their argument checks to no rows)
    assert dsa.dsa_cache_append_q8(_pb(dsa, "chunk", 0, 4096), *[FAKE] * 5, None, 0) == dsa.DSA_OK
