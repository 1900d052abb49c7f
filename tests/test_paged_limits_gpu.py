"""The paged-cache operators at the edges of what they take: row ranges and lengths out of their limits, values at the ends
of their types' ranges, handles of odd strides, what a call does to torch's own state."""
import numpy as np
import pytest
import torch

import paged_ref as R

pytestmark = pytest.mark.gpu
ms = pytest.importorskip("decoder_only_transformer_int4_b200")

U = 2.0 ** -23


def _same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---- the append leaves out what the attention leaves out --------------------------------------

BAD_RANGES = {
    # name: (lens, row_start, sequences left out, rows of no sequence)
    "past the rows": ([40, 40, 40], [0, 2, 4, 9], [2], []),
    "past the rows, from a row that is not there": ([40, 40, 40], [0, 2, 6, 9], [2], []),
    "decreasing": ([40, 40, 40], [0, 4, 3, 6], [1], []),
    "negative": ([40, 40, 40], [-2, 2, 4, 6], [0], []),
    "rows before the first sequence": ([40, 40, 40], [2, 3, 4, 6], [], [0, 1]),
    "length past the capacity": ([40, 50, 40], [0, 2, 4, 6], [1], []),
    "length below zero": ([40, -1, 40], [0, 2, 4, 6], [1], []),
    "more rows than positions": ([40, 2, 40], [0, 1, 4, 6], [1], []),
    "length past the capacity of a sequence without rows": ([40, 50, 40], [0, 3, 3, 6], [1], []),
}


@pytest.mark.parametrize("kq,kkv", R.PAIRS)
@pytest.mark.parametrize("case", list(BAD_RANGES))
@pytest.mark.parametrize("heads,skew", [(4, 0), (4, 1), (0, 0)])
def test_append_leaves_out_bad_sequences(kq, kkv, case, heads, skew):
    lens, start, bad, loose = BAD_RANGES[case]
    hk, hd, rows = 2, 64, 6
    pages = R.Pages([40, 40, 40], hk, 16, hd, kkv, seed=401)         # 3 pages each: 48 positions
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = pages.cuda(ms, status, lens=lens)
    k0, v0 = pages.dk.clone(), pages.dv.clone()
    g = torch.Generator().manual_seed(402)
    buf = torch.randn((rows, (heads + 2 * hk) * hd + skew), generator=g).to(R.TYPES[kq]).cuda()
    x = buf.as_strided((rows, heads + 2 * hk, hd), (buf.shape[1], hd, 1), skew)
    f = torch.tensor([1e4 ** (-2 * j / hd) for j in range(hd // 2)], dtype=torch.float64)
    out = torch.full((rows, heads, hd), 7.0, dtype=x.dtype, device="cuda") if heads else None
    ms.rope_append_paged(kv, x[:, :heads] if heads else None, x[:, heads:heads + hk], x[:, heads + hk:],
                         torch.tensor(start, dtype=torch.int32).cuda(), f.cuda(), out=out)
    if bad:
        with pytest.raises(ms.MsError) as e:
            ms.op_status(status)
        assert e.value.status == ms.MS_ERR_SHAPE
    else:
        ms.op_status(status)
    # a row belongs to the sequence whose end is the first behind it
    at = {}
    for t in range(rows):
        b = sum(s <= t for s in start[1:])
        if b < 3 and b not in bad and t >= start[b]:
            at[t] = (b, lens[b] - (start[b + 1] - start[b]) + t - start[b])
    assert not set(at) & set(loose)
    xs = R.f64(x)
    for t, (b, pos) in at.items():
        want = R.rotate(xs[t:t + 1, :heads + hk], [pos], f.numpy(), False, 1.0)[0]
        p, i = int(pages.table[b, pos // 16]), pos % 16
        mag = np.sqrt((xs[t, :heads + hk] ** 2).sum(-1, keepdims=True))
        # as in test_paged_gpu.py: sines, products and the sum are off by 8 * 2^-24 of the pair's size, then one rounding
        tol = lambda kind, y, m: R.half_step(kind) * np.abs(y) + 8 * 2.0 ** -24 * m + (2.0 ** -25 if kind == "f16" else 0)  # noqa: E731
        assert np.all(np.abs(R.f64(pages.dk[p, :, i]) - want[heads:]) <= tol(kkv, want[heads:], mag[heads:]))
        assert np.array_equal(R.f64(pages.dv[p, :, i]), R.f64(x[t, heads + hk:].to(R.TYPES[kkv])))
        if heads:
            assert np.all(np.abs(R.f64(out[t]) - want[:heads]) <= tol(kq, want[:heads], mag[:heads]))
        pages.dk[p, :, i], pages.dv[p, :, i] = k0[p, :, i], v0[p, :, i]
    assert _same(pages.dk, k0) and _same(pages.dv, v0)              # nothing else was written
    if heads:
        assert all(bool((out[t] == 7.0).all()) for t in range(rows) if t not in at)


# ---- fp32 queries on a half cache ---------------------------------------------------------------

@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** 126, 2.0 ** 118, 2.0 ** -105, 2.0 ** -126])
def test_attention_of_queries_at_the_ends_of_fp32(hd, size):
    # powers of two: the scores are those of the unscaled queries
    pages = R.Pages([200, 70], 1, 16, hd, "f16", seed=411)
    g = torch.Generator().manual_seed(412)
    q = torch.rand((3, 2, hd), generator=g) * 2 - 1                    # below 2 in size: q * size below 2^127
    big = (q * size).cuda()
    x = big.cpu().double().numpy() / size                              # what is left of them where they are subnormal
    scale = 2.0 / size if size <= 2.0 ** 126 else None
    got = R.f64(ms.attn_paged(pages.cuda(ms), big, R.starts([1, 2]).cuda(), 2, scale=scale))
    ref, A, spread, _ = R.attention(pages, torch.from_numpy(x), [1, 2], 2.0)
    T = np.array([200, 70, 70])[:, None]
    # as in test_paged_gpu.py: (hd + 16) U of the products' sum for a score, 2^-21 for the pairs, 2 T U for the sums
    tol = R.half_step("f32") * np.abs(ref) + A * (2 * (hd + 17) * U * spread + 8 * U + 2.0 ** -21 + 2 * T * U)[..., None]
    assert np.all(np.abs(got - ref) <= tol), np.abs(got - ref).max()


@pytest.mark.parametrize("kq,kkv", [("f32", "f16"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("T", [9, 16, 200, 1500])
@pytest.mark.parametrize("nats", [10, 17, 24, 30, 45, 70])
@pytest.mark.parametrize("group", [1, 12, 28])
def test_attention_where_the_heaviest_position_holds_nothing(kq, kkv, hd, T, nats, group):
    """One position leads all others by `nats` and its v is 0: the result is made of probabilities e^-nats and below alone."""
    pages = R.Pages([T], 1, 16, hd, kkv, seed=421)
    g = torch.Generator().manual_seed(422)
    lead = T // 3
    for i in range(T):
        p, j = int(pages.table[0, i // 16]), i % 16
        pages.k[p, 0, j] = 0.0
        # multiples of 1/4 below 16: exact in every type, and so are the scores before the factor log2 e
        pages.k[p, 0, j, 0] = 0.0 if i == lead else -nats - 0.25 * int(torch.randint(0, 16, (1,), generator=g))
        if i == lead:
            pages.v[p, 0, j] = 0.0
    q = torch.zeros((1, group, hd))
    q[..., 0] = 1.0
    q = q.to(R.TYPES[kq])
    got = R.f64(ms.attn_paged(pages.cuda(ms), q.cuda(), R.starts([1]).cuda(), 1, scale=1.0))
    ref, A, spread, _ = R.attention(pages, q, [1], 1.0)
    # a score's exact product takes two roundings (the factor and the product, 2^-24 each) and a third where the reference is
    # subtracted, so a probability is off by 2 * 3/2 U |s|; exp2 4 U above and below; the pairs 2^-21 or 2^-17; two sums of T
    tol = R.half_step(kq) * np.abs(ref) + A * (3 * U * spread + 8 * U + (2.0 ** -17 if kkv == "bf16" else 2.0 ** -21) + 2 * T * U)[..., None]
    assert np.all(np.abs(got - ref) <= tol), (np.abs(got - ref) / np.maximum(A, 1e-300)).max()

@pytest.mark.parametrize("kq,kkv,v", [("bf16", "bf16", 2.0 ** 91), ("f32", "f32", 2.0 ** 91), ("f32", "f16", 65504.0), ("f16", "f16", 65504.0)])
def test_attention_of_the_largest_values(kq, kkv, v):
    # the sums over 3000 positions, before they are divided, stay finite (an fp16 result may round up to infinity)
    T = 3000
    pages = R.Pages([T], 1, 64, 64, kkv, seed=461)
    pages.v = torch.where(torch.isnan(pages.v), pages.v, torch.full_like(pages.v, v))
    q = torch.ones((1, 4, 64)).to(R.TYPES[kq])
    got = R.f64(ms.attn_paged(pages.cuda(ms), q.cuda(), R.starts([1]).cuda(), 1))
    # all v are the same: the two sums over T positions, exp2 twice, the pairs; then one rounding
    rel = R.half_step(kq) + 2 * T * U + 8 * U + (2.0 ** -17 if kkv == "bf16" else 2.0 ** -21)
    assert np.all(np.isfinite(got) | (kq == "f16")) and np.all(np.abs(np.minimum(got, v) - v) <= rel * v)


# ---- verification ---------------------------------------------------------------------------------

@pytest.mark.parametrize("where", ["target", "draft"])
@pytest.mark.parametrize("V", [50, 20000])
def test_verification_flags_rows_with_nan(where, V):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(431)
    target = torch.softmax(torch.randn((3, V), generator=g), 1).cuda()
    draft = torch.softmax(torch.randn((1, V), generator=g), 1).cuda()
    (target if where == "target" else draft)[0, 7] = float("nan")
    tok = torch.tensor([3], dtype=torch.int32, device="cuda")
    ua = torch.full((1,), 1 - 2.0 ** -24, device="cuda")
    draft[0, 3] = 1.0                                                   # refused: u q >= p
    acc, out = ms.verify_draft(target, draft, tok, R.starts([1, 0]).cuda(), 1, ua, torch.full((2,), 0.5, device="cuda"), status)
    with pytest.raises(ms.MsError) as e:
        ms.op_status(status)
    assert e.value.status == ms.MS_ERR_TOKEN_RANGE
    assert acc.cpu().tolist() == [0, 0] and out.cpu()[0].tolist() == [-1, -1] and out[1, 0].item() >= 0


# ---- how the attention's work is laid out -------------------------------------------------------------

@pytest.mark.parametrize("kq,kkv,group", [("f16", "f16", 28), ("bf16", "bf16", 32), ("f32", "f16", 25), ("f32", "f16", 24)])
def test_attention_plans_no_more_ctas_than_fit(kq, kkv, group):
    """The workspace holds two slots of (hd + 2) floats a row for each CTA of the grid.  Three CTAs of 128 threads an SM leave 168
    registers a thread; the kernels of these shapes (24 and more rows of 64 elements in registers) need more, so two fit."""
    hd, page, batch = 64, 256, 64
    table = torch.zeros((batch, 64), dtype=torch.int32, device="cuda")
    k = torch.zeros((1, 1, page, hd), dtype=R.TYPES[kkv], device="cuda")
    kv = ms.PagedKV(k, k.clone(), table, torch.zeros(batch, dtype=torch.int32, device="cuda"))
    rows = -(-group // 8) * 8
    ctas = ms.attn_paged_workspace(kv, R.TYPES[kq], group, 1) / (2 * rows * (hd + 2) * 4)
    assert round(ctas) == 2 * torch.cuda.get_device_properties(0).multi_processor_count


# ---- torch's side of a call ---------------------------------------------------------------------------

def test_refused_calls_allocate_nothing():
    pages = R.Pages([40, 3], 2, 16, 64, "f16", seed=441, spare=6)
    kv = pages.cuda(ms)
    w = torch.zeros((2, 2, kv.capacity), device="cuda")
    dst = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    q, st = torch.zeros((2, 6, 64), dtype=torch.float16, device="cuda"), R.starts([1, 1]).cuda()
    for call, code in ((lambda: ms.evict_paged(kv, w, dst, 1 << 20, first=(1 << 20) + 1), ms.MS_ERR_SHAPE),
                       (lambda: ms.evict_paged(kv, w[..., :16].contiguous(), dst, 1 << 20), ms.MS_ERR_SHAPE),
                       (lambda: ms.attn_paged(kv, q.expand(2, 6, 64).bfloat16().repeat(1 << 10, 1, 1), st, 1), ms.MS_ERR_UNSUPPORTED),
                       (lambda: ms.attn_paged(kv, q[:, :5].repeat(1 << 10, 1, 1), st, 1), ms.MS_ERR_SHAPE)):
        torch.cuda.synchronize()
        n0 = torch.cuda.memory_stats()["allocation.all.allocated"]
        with pytest.raises(ms.MsError) as e:
            call()
        assert e.value.status == code
        made = torch.cuda.memory_stats()["allocation.all.allocated"] - n0
        assert made <= 2, made                                          # the arguments of the call alone


def test_calls_count_as_writes():
    """Pages, weights and outputs that a call writes carry a new version, so that autograd notices."""
    pages = R.Pages([40], 1, 16, 64, "f32", seed=451, spare=8)
    kv = pages.cuda(ms)
    x, st = torch.randn((1, 1, 64), device="cuda"), R.starts([1]).cuda()
    w, out = torch.zeros((1, 1, kv.capacity), device="cuda"), torch.empty((1, 1, 64), device="cuda")
    dst = torch.tensor([pages.free[:1]], dtype=torch.int32, device="cuda")

    def versions():
        return [t._version for t in (pages.dk, pages.dv, w, out)]

    for call, written in ((lambda: ms.rope_append_paged(kv, x, x, x, st, None, out=out), (1, 1, 0, 1)),
                          (lambda: ms.rope_append_paged(kv, None, x, x, st, None), (1, 1, 0, 0)),
                          (lambda: ms.attn_paged(kv, x, st, 1, weights=w, out=out), (0, 0, 1, 1)),
                          (lambda: ms.attn_paged(kv, x, st, 1), (0, 0, 0, 0)),
                          (lambda: ms.evict_paged(kv, w, dst, 16), (1, 1, 0, 0)),
                          (lambda: ms.evict_paged(kv, w, dst, 16, weights_out=w), (1, 1, 1, 0))):
        before = versions()
        call()
        assert tuple(b > a for a, b in zip(before, versions())) == tuple(map(bool, written))
    with torch.inference_mode():                                        # such tensors have no version
        w2 = torch.zeros((1, 1, kv.capacity), device="cuda")
        ms.attn_paged(kv, x, st, 1, weights=w2)


def test_a_cache_of_one_page_may_have_any_stride_there():
    big = torch.randn((2, 1, 16, 64), device="cuda")
    k, v = big[:1].as_strided((1, 1, 16, 64), (5000, 77, 64, 1)), big[1:]
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.full((1,), 16, dtype=torch.int32, device="cuda")
    q = torch.randn((1, 1, 64), device="cuda")
    got = ms.attn_paged(ms.PagedKV(k, v, table, lens), q, R.starts([1]).cuda(), 1)
    want = ms.attn_paged(ms.PagedKV(big[:1], v, table, lens), q, R.starts([1]).cuda(), 1)
    assert torch.equal(got, want)
    for bad in (big[1:].expand(1, 1, 16, 64).transpose(2, 3), big.half()[1:], big):
        with pytest.raises(ValueError):
            ms.PagedKV(k, bad, table, lens)
