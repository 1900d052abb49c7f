"""What the paged-cache entry points refuse, found on the host before any device work.  No GPU needed."""
import ctypes

import pytest
import torch

ms = pytest.importorskip("decoder_only_transformer_int4_b200")
L = ms._lib
P = 4096          # a 16-byte aligned address that nothing reads


def kv(**change):
    f = dict(k=P, v=P, elem=ms.MS_ELEM_F16, n_pages=8, page_size=16, n_kv_heads=2, head_dim=64, page_stride=2048, table=P,
             max_pages=4, batch=3, lens=P, status=None)
    f.update(change)
    return ctypes.byref(ms.PagedKVStruct(**f))


def rope(cache=None, q=P, ldq=512, k=P, ldk=128, v=P, ldv=128, elem=ms.MS_ELEM_F16, rows=5, heads=8, start=P, positions=None, freq=P, rot=64,
         mscale=1.0, out=P, ldo=512):
    return L.ms_op_rope_append_paged(cache or kv(), q, ldq, k, ldk, v, ldv, elem, rows, heads, start, positions, freq, rot, 0, mscale, out, ldo,
                                     None)


def attn(cache=None, q=P, ldq=512, elem=ms.MS_ELEM_F16, rows=5, most=4, heads=8, scale=0.125, start=P, out=P, ldo=512, weights=None, ldw=0,
         ws=P, size=1 << 30):
    return L.ms_op_attn_paged(cache or kv(), q, ldq, elem, rows, most, heads, scale, start, out, ldo, weights, ldw, ws, size, None)


def evict(cache=None, weights=P, ldw=64, dst=P, pages=2, keep=32, first=4, recent=8, kept=P, out=2 * P, ldo=64, lens=2 * P):
    return L.ms_op_evict_paged(cache or kv(), weights, ldw, dst, pages, keep, first, recent, kept, out, ldo, lens, None)


def verify(target=P, ldt=100, draft=P, ldd=100, tokens=P, start=P, rows=6, batch=2, most=4, vocab=100, ua=P, us=P, accepted=P, out=P):
    return L.ms_op_verify_draft(target, ldt, draft, ldd, tokens, start, rows, batch, most, vocab, ua, us, accepted, out, None, None)


INVALID, SHAPE, UNSUPPORTED = ms.MS_ERR_INVALID_ARG, ms.MS_ERR_SHAPE, ms.MS_ERR_UNSUPPORTED
CACHES = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(elem=3), INVALID),
          (dict(elem=-1), INVALID), (dict(table=P + 2), INVALID), (dict(lens=P + 1), INVALID), (dict(status=P + 2), INVALID), (dict(k=P + 8), INVALID), (dict(v=P + 2), INVALID), (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE),
          (dict(page_size=0), SHAPE), (dict(page_size=-16), SHAPE), (dict(head_dim=80), SHAPE), (dict(n_kv_heads=0), SHAPE),
          (dict(n_kv_heads=5000), SHAPE), (dict(n_pages=0), SHAPE), (dict(batch=0), SHAPE), (dict(batch=1025), SHAPE), (dict(max_pages=0), SHAPE),
          (dict(max_pages=1 << 26), SHAPE), (dict(page_stride=2047), SHAPE), (dict(page_stride=2052), SHAPE), (dict(page_stride=-2048), SHAPE),
          (dict(page_stride=1 << 60), SHAPE)]


@pytest.mark.parametrize("change,want", CACHES)
def test_caches_that_are_refused(change, want):
    assert rope(kv(**change)) == want and ms.last_error().startswith("ms_op_rope_append_paged")
    assert attn(kv(**change)) == want and ms.last_error().startswith("ms_op_attn_paged")
    assert evict(kv(**change)) == want and ms.last_error().startswith("ms_op_evict_paged")
    assert L.ms_op_attn_paged_workspace(kv(**change), ms.MS_ELEM_F16, 8, 1, 0) == 0


def test_no_cache_and_no_status_word():
    assert L.ms_op_rope_append_paged(None, P, 512, P, 128, P, 128, 1, 5, 8, P, None, P, 64, 0, 1.0, P, 512, None) == INVALID
    assert L.ms_op_attn_paged(None, P, 512, 1, 5, 4, 8, 0.125, P, P, 512, None, 0, P, 1 << 30, None) == INVALID
    assert L.ms_op_evict_paged(None, P, 64, P, 2, 32, 4, 8, P, P, 64, P, None) == INVALID
    assert L.ms_op_status(None, None) == INVALID and L.ms_op_status(P + 2, None) == INVALID


@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), SHAPE), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(start=None), INVALID), (dict(freq=None), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(elem=ms.MS_ELEM_BF16), UNSUPPORTED), (dict(elem=7), UNSUPPORTED),
    (dict(rot=-2), SHAPE), (dict(rot=63), SHAPE), (dict(rot=66), SHAPE), (dict(heads=0), SHAPE), (dict(heads=1 << 20), SHAPE), (dict(ldq=511), SHAPE),
    (dict(ldk=127), SHAPE), (dict(ldv=0), SHAPE), (dict(ldo=-512), SHAPE), (dict(ldk=1 << 50), SHAPE), (dict(k=P + 1), INVALID),
    (dict(freq=P + 4), INVALID), (dict(start=P + 2), INVALID), (dict(positions=P + 1), INVALID)])
def test_rope_refuses(change, want):
    assert rope(**change) == want


def test_rope_of_no_rows_is_nothing():
    assert rope(rows=0) == ms.MS_OK and rope(rows=0, q=None, out=None, k=None, v=None) == ms.MS_OK


@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), SHAPE), (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(start=None), INVALID), (dict(ws=None), INVALID),
    (dict(ws=P + 128), INVALID), (dict(elem=ms.MS_ELEM_BF16), UNSUPPORTED), (dict(most=0), SHAPE), (dict(most=65), SHAPE), (dict(heads=7), SHAPE),
    (dict(heads=0), SHAPE), (dict(heads=2 * 257, ldq=1 << 20, ldo=1 << 20), SHAPE), (dict(ldq=500), SHAPE), (dict(ldo=0), SHAPE),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(weights=P, ldw=63), SHAPE), (dict(weights=P + 2, ldw=64), INVALID),
    (dict(q=P + 1), INVALID), (dict(start=P + 2), INVALID)])
def test_attention_refuses(change, want):
    assert attn(**change) == want
    if set(change) <= {"most", "heads", "elem"}:
        f = dict(elem=ms.MS_ELEM_F16, most=4, heads=8, **{})
        f.update(change)
        assert L.ms_op_attn_paged_workspace(kv(), f["elem"], f["heads"], f["most"], 0) == 0


def test_attention_refuses_pairs_of_types_without_a_kernel():
    ok = {(0, 0), (0, 1), (1, 1), (2, 2)}
    for q in range(3):
        for c in range(3):
            if (q, c) not in ok:
                assert attn(kv(elem=c, page_stride=2048), elem=q) == UNSUPPORTED
                assert rope(kv(elem=c, page_stride=2048), elem=q) == UNSUPPORTED


def test_attention_refuses_sizes_whose_tiles_do_not_fit_31_bits():
    big = kv(max_pages=1 << 20, page_size=512, page_stride=1 << 16, batch=1024)
    assert attn(big, heads=64, ldq=1 << 20, ldo=1 << 20, most=64) == SHAPE


@pytest.mark.parametrize("change,want", [
    (dict(weights=None), INVALID), (dict(dst=None), INVALID), (dict(kept=None), INVALID), (dict(out=None), INVALID), (dict(lens=None), INVALID),
    (dict(lens=P), INVALID), (dict(keep=0), SHAPE), (dict(first=-1), SHAPE), (dict(recent=-1), SHAPE), (dict(first=20, recent=13), SHAPE),
    (dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), SHAPE), (dict(pages=0), SHAPE), (dict(ldw=63), SHAPE), (dict(ldo=31), SHAPE), (dict(keep=100, ldo=63), SHAPE),
    (dict(out=P, ldo=65), SHAPE), (dict(weights=P + 2), INVALID), (dict(dst=P + 1), INVALID), (dict(kept=P + 2), INVALID), (dict(out=P + 2), INVALID),
    (dict(lens=P + 6), INVALID)])
def test_eviction_refuses(change, want):
    assert evict(**change) == want


@pytest.mark.parametrize("change,want", [
    (dict(target=None), INVALID), (dict(start=None), INVALID), (dict(us=None), INVALID), (dict(accepted=None), INVALID), (dict(out=None), INVALID),
    (dict(tokens=None), INVALID), (dict(ua=None), INVALID), (dict(rows=-1), SHAPE), (dict(batch=0), SHAPE), (dict(batch=(1 << 20) + 1), SHAPE),
    (dict(vocab=0), SHAPE), (dict(most=-1), SHAPE), (dict(most=257), SHAPE), (dict(ldt=99), SHAPE), (dict(ldd=99), SHAPE), (dict(ldt=1 << 50), SHAPE),
    (dict(target=P + 2), INVALID), (dict(draft=P + 2), INVALID), (dict(tokens=P + 1), INVALID), (dict(start=P + 2), INVALID), (dict(ua=P + 2), INVALID),
    (dict(us=P + 2), INVALID), (dict(accepted=P + 2), INVALID), (dict(out=P + 2), INVALID)])
def test_verification_refuses(change, want):
    assert verify(**change) == want


def test_python_calls_refuse_tensors_of_the_cpu_and_things_that_are_none():
    t = torch.zeros(2, 1, 16, 64)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ms.PagedKV(t, t, i, i[0])
    with pytest.raises(ValueError, match="expected a tensor"):
        ms.PagedKV(t, None, i, i[0])
    with pytest.raises(ValueError, match="CUDA"):
        ms.verify_draft(torch.ones(3, 5), None, i[0], torch.tensor([0, 1], dtype=torch.int32), 1, torch.zeros(1), torch.zeros(1))
    with pytest.raises(ValueError):
        ms._paged.rope("x", *[None] * 9)          # not a cache
    with pytest.raises(TypeError):
        ms._paged.attn(1, 2)
