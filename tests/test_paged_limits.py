"""The context limit of attention over every prior key of the paged caches: 131072 keys, whatever the
rows (checked before any device is touched, with addresses that are never read)."""
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
