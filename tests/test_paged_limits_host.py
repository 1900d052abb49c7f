"""Sizes that the paged-cache entry points refuse on the host.  No GPU needed."""
from test_paged_host import P, SHAPE, attn, kv, ms, rope, verify

L = ms._lib


def test_attention_refuses_as_many_tiles_as_its_counts_could_not_pass():
    # 993 sequences of 2162622 tiles of 64 positions are 2^31 - 2: the kernel rounds the count up to whole runs for its CTAs,
    # which has to stay below 2^31 as well
    huge = dict(max_pages=2162622, page_size=64, page_stride=1 << 12, batch=993, n_kv_heads=1)
    assert 993 * 2162622 == 2 ** 31 - 2
    assert attn(kv(**huge), heads=1, ldq=64, ldo=64, most=1, size=1 << 62) == SHAPE
    assert L.ms_op_attn_paged_workspace(kv(**huge), ms.MS_ELEM_F16, 1, 1, 0) == 0


MOST = 1 << 30


def test_rows_and_vocabularies_past_the_kernels_indices_are_refused():
    for n in (MOST + 1, 2 ** 31 - 1):
        assert rope(rows=n) == SHAPE and attn(rows=n) == SHAPE and verify(rows=n) == SHAPE
        assert verify(vocab=n, ldt=1 << 32, ldd=1 << 32) == SHAPE


def test_in_place_needs_the_same_row_stride():
    # another stride would let one row's result overwrite another row's input
    assert rope(out=P, ldo=1024) == SHAPE and "in place" in ms.last_error()
    assert attn(out=P, ldo=1024) == SHAPE and "in place" in ms.last_error()
