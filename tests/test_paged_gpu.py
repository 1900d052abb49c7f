"""The paged-cache operators against plain 64-bit restatements (tests/paged_ref.py).

Tolerances are counted, not fitted.  u = 2^-23 bounds one fp32 step of a tensor-core sum (which may truncate).

Attention.  A score is a sum of hd products, off by at most (hd + 16) u of the sum of their magnitudes: hd for the
additions, 16 for the operands (fp32 ones enter with 21 bits or more: 2 * 2^-21 = 8 u in all, and the scale and the
base change 4 more).  That moves a probability by twice as much relatively (numerator and denominator), exp2 by 4 u,
and the subtraction of the maximum by |score| u (below the magnitudes' sum).  The probabilities enter the second product with 2^-17
(bf16 pairs) or 2^-21; the two sums over T positions add 2 T u.  Then one rounding to the type.
"""
import numpy as np
import pytest
import torch

import paged_ref as R

pytestmark = pytest.mark.gpu
ms = pytest.importorskip("decoder_only_transformer_int4_b200")

U = 2.0 ** -23
LENS = [1, 15, 16, 17, 0, 63, 64, 65, 130, 300]


def _attn_tol(kind_q, kind_kv, hd, T, out, A, spread):
    p = 2 * ((hd + 16) * U * spread + spread * U) + 8 * U
    second = 2.0 ** -17 if kind_kv == "bf16" else 2.0 ** -21
    return R.half_step(kind_q) * np.abs(out) + A * (p + second + 2 * T * U)[..., None] + 1e-30 + \
        (2.0 ** -25 if kind_q == "f16" else 0)


def _check_attn(kind_q, kind_kv, hd, hk, group, page, lens, counts, seed, weights=False, scale=None, q_scale=1.5, most=None,
                pages=None):
    pages = R.Pages(lens, hk, page, hd, kind_kv, seed) if pages is None else pages
    rows, H = sum(counts), hk * group
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn((rows + 2, H, hd), generator=g) * q_scale).to(R.TYPES[kind_q])
    scale = hd ** -0.5 if scale is None else scale
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = pages.cuda(ms, status)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    w = w0 = None
    if weights:
        w0 = torch.rand((len(lens), hk, kv.capacity + 3), generator=g)
        w = w0.cuda()
    ms.attn_paged(kv, q.cuda(), R.starts(counts).cuda(), most or max(1, max(counts)), scale=scale, weights=w, out=out)
    ms.op_status(status)
    ref, A, spread, rw = R.attention(pages, q[:rows], counts, scale)
    got = R.f64(out)
    assert np.all(got[rows:] == 7.0)          # rows behind the last sequence are left as they were
    T = np.repeat(np.array(lens), counts)[:, None]
    assert np.all(np.isfinite(got[:rows]))
    err, tol = np.abs(got[:rows] - ref), _attn_tol(kind_q, kind_kv, hd, T, ref, A, spread)
    assert np.all(err <= tol), (err.max(), (err / tol).max())
    if weights:
        gw, r = R.f64(w), 0
        for b, (t, n) in enumerate(zip(lens, counts)):
            assert np.array_equal(gw[b, :, t:], R.f64(w0)[b, :, t:])
            sp = spread[r:r + n].max() if n else 0.0
            rel = 2 * (hd + 17) * U * sp + (8 + 2 * t + n * group) * U
            was = R.f64(w0)[b, :, :t]
            assert np.all(np.abs(gw[b, :, :t] - was - rw[b]) <= rel * rw[b] + U * (was + rw[b])), b
            r += n
    return got[:rows]


@pytest.mark.parametrize("kq,kkv", R.PAIRS)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 7])
def test_attention_one_row(kq, kkv, hd, group):
    _check_attn(kq, kkv, hd, 2, group, 16, LENS, [1] * len(LENS), seed=11 + group, weights=True)


@pytest.mark.parametrize("kq,kkv", R.PAIRS)
@pytest.mark.parametrize("hd,page", [(64, 32), (128, 64)])
@pytest.mark.parametrize("group,most", [(4, 5), (8, 8), (1, 16), (20, 3)])
def test_attention_drafted_rows(kq, kkv, hd, page, group, most):
    # row counts 0 .. most, among them more rows than positions (rows that see nothing)
    counts = [min(most, c) for c in (most, 1, 0, 3, 2, most, most - 1, 2, most, most)]
    _check_attn(kq, kkv, hd, 2, group, page, LENS, counts, seed=31 + group, weights=True, most=most)


@pytest.mark.parametrize("kq,kkv", R.PAIRS)
def test_attention_is_split_and_joined(kq, kkv):
    # one sequence over many CTAs, next to short ones
    _check_attn(kq, kkv, 64, 1, 3, 64, [2500, 5, 700], [1, 1, 2], seed=51, weights=True)
    _check_attn(kq, kkv, 128, 2, 2, 256, [1500], [4], seed=52)


@pytest.mark.parametrize("kq,kkv", R.PAIRS)
def test_attention_peaked_and_flat_scores(kq, kkv):
    _check_attn(kq, kkv, 64, 1, 4, 16, [200, 64], [1, 2], seed=61, q_scale=30.0)
    _check_attn(kq, kkv, 64, 1, 4, 16, [200, 64], [1, 2], seed=62, q_scale=1e-3)
    _check_attn(kq, kkv, 64, 1, 4, 16, [200, 64], [1, 2], seed=63, scale=0.0)
    _check_attn(kq, kkv, 64, 1, 4, 16, [200, 64], [1, 2], seed=64, scale=-0.25)


@pytest.mark.parametrize("kq,kkv", R.PAIRS)
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_attention_rows_ignore_later_drafts(kq, kkv, what):
    # the last draft's k and v are not finite: only the row that sees it may notice
    for T in (65, 64, 40):
        pages = R.Pages([T], 1, 16, 64, kkv, seed=71)
        i = T - 1
        p = int(pages.table[0, i // 16])
        pages.k[p, :, i % 16] = what
        pages.v[p, :, i % 16, ::3] = what
        q = torch.randn((3, 2, 64), generator=torch.Generator().manual_seed(5)).to(R.TYPES[kq])
        kv = pages.cuda(ms)
        got = R.f64(ms.attn_paged(kv, q.cuda(), R.starts([3]).cuda(), 3))
        pages.lens = [T - 1]
        ref, A, spread, _ = R.attention(pages, q[:2], [2], 0.125)
        tol = _attn_tol(kq, kkv, 64, np.array([[T]]), ref, A, spread)
        assert np.all(np.abs(got[:2] - ref) <= tol)
        assert not np.all(np.isfinite(got[2]))


def test_attention_flags_bad_device_data_and_leaves_it_out():
    lens = [40, 40, 40, 40, 40]
    pages = R.Pages(lens, 1, 16, 64, "f32", seed=81)
    q = torch.randn((5, 2, 64), generator=torch.Generator().manual_seed(6))
    ref, A, spread, _ = R.attention(pages, q, [1] * 5, 0.125)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = R.starts([1] * 5)
    for what in ("len", "negative", "page", "rows"):
        lens2, st2 = list(lens), start.clone()
        if what == "len":
            lens2[2] = 49
        if what == "negative":
            lens2[2] = -1
        kv = pages.cuda(ms, status, lens=lens2)
        if what == "page":
            pages.dtable[2, 1] = pages.n_pages
        if what == "rows":
            st2[5] = 9
        out = torch.full(q.shape, 7.0, device="cuda")
        ms.attn_paged(kv, q.cuda(), st2.cuda(), 1, out=out)
        with pytest.raises(ms.MsError) as e:
            ms.op_status(status)
        assert e.value.status == ms.MS_ERR_SHAPE
        ms.op_status(status)                      # cleared
        got, bad = R.f64(out), 4 if what == "rows" else 2
        good = [i for i in range(5) if i != bad]
        assert np.all(np.abs(got - ref)[good] <= _attn_tol("f32", "f32", 64, np.full((5, 1), 40), ref, A, spread)[good])
        if what != "page":
            assert np.all(got[bad] == 7.0)


def test_attention_in_a_graph_follows_lengths_and_tables():
    pages = R.Pages([90, 33, 120], 2, 16, 64, "f16", seed=91, extra=40)
    H = 8
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = pages.cuda(ms, status)
    q = torch.randn((3, H, 64), generator=torch.Generator().manual_seed(7)).cuda()
    st = R.starts([1, 1, 1]).cuda()
    out = torch.zeros_like(q)
    w = torch.zeros((3, 2, kv.capacity), device="cuda")
    ws = torch.empty(ms.attn_paged_workspace(kv, torch.float32, H, 1, True), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ms.attn_paged(kv, q, st, 1, out=out, weights=w, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ms.attn_paged(kv, q, st, 1, out=out, weights=w, workspace=ws)
    for lens in ([90, 33, 120], [1, 0, 119], [64, 17, 3]):
        pages.dlens.copy_(torch.tensor(lens, dtype=torch.int32))
        q.normal_()
        w.zero_()
        graph.replay()
        ms.op_status(status)
        pages.lens = lens
        ref, A, spread, rw = R.attention(pages, q, [1, 1, 1], 0.125)
        tol = _attn_tol("f32", "f16", 64, np.array(lens)[:, None], ref, A, spread)
        assert np.all(np.abs(R.f64(out) - ref) <= tol)


# ---- rotary positions and append -----------------------------------------------------------

def _freqs(rot, base=1e4):
    return torch.tensor([base ** (-2 * j / rot) for j in range(rot // 2)], dtype=torch.float64)


def _rope_tol(kind, y, x, mscale):
    """sincospif is off by at most 2 * 2^-24 and its argument by 2^-24; with the factor, two products and a sum: 8 * 2^-24 of
    the pair's magnitude; then one rounding."""
    mag = np.abs(x) * 0 + np.sqrt((x ** 2).sum(-1, keepdims=True))
    return R.half_step(kind) * np.abs(y) + 8 * 2.0 ** -24 * abs(mscale) * mag + (2.0 ** -25 if kind == "f16" else 1e-40)


@pytest.mark.parametrize("kq,kkv", R.PAIRS)
@pytest.mark.parametrize("hd,rot", [(64, 64), (128, 128), (128, 64), (64, 30), (64, 2), (128, 96), (64, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_append(kq, kkv, hd, rot, interleaved):
    H, hk, page = 6, 2, 16
    counts = [1, 0, 20, 3, 33]
    lens = [17, 40, 20, 63, 70]
    pages = R.Pages(lens, hk, page, hd, kkv, seed=101)
    rows = sum(counts)
    g = torch.Generator().manual_seed(102)
    fused = torch.randn((rows + 3, (H + 2 * hk), hd), generator=g).to(R.TYPES[kq])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for shift, positions in ((0, None), (100000, True)):
        kv = pages.cuda(ms, status)
        d = fused.cuda()
        before_k, before_v = f_all(pages.dk), f_all(pages.dv)
        out = torch.full((rows + 3, H, hd), 7.0, dtype=d.dtype, device="cuda")
        pos = np.concatenate([np.arange(t - n, t) for t, n in zip(lens, counts)]) + shift
        dp = torch.tensor(np.concatenate([pos, [0, 0, 0]]), dtype=torch.int32).cuda() if positions else None
        f = _freqs(rot) if rot else None
        mscale = 1.0 if not positions else 1.25
        ms.rope_append_paged(kv, d[:, :H], d[:, H:H + hk], d[:, H + hk:], R.starts(counts).cuda(),
                             None if f is None else f.cuda(), interleaved=interleaved, mscale=mscale, positions=dp, out=out)
        ms.op_status(status)
        x = R.f64(fused[:rows])
        fr = f.numpy() if rot else np.zeros(0)
        want = R.rotate(x[:, :H + hk], pos, fr, interleaved, mscale)
        got = R.f64(out)
        assert np.all(got[rows:] == 7.0)
        assert np.all(np.abs(got[:rows] - want[:, :H]) <= _rope_tol(kq, want[:, :H], x[:, :H], mscale))
        gk, gv = f_all(pages.dk), f_all(pages.dv)
        r = 0
        for b, (t, n) in enumerate(zip(lens, counts)):
            for i in range(t - n, t):
                p = int(pages.table[b, i // page])
                tol = _rope_tol(kkv, want[r, H:], x[r, H:H + hk], mscale)
                assert np.all(np.abs(gk[p, :, i % page] - want[r, H:]) <= tol)
                assert np.array_equal(gv[p, :, i % page], R.f64(fused[r, H + hk:].to(R.TYPES[kkv])))
                before_k[p, :, i % page], before_v[p, :, i % page] = gk[p, :, i % page], gv[p, :, i % page]
                r += 1
        assert np.array_equal(gk, before_k, equal_nan=True) and np.array_equal(gv, before_v, equal_nan=True)


def f_all(t):
    return R.f64(t)


def test_rope_in_place_unaligned_and_far():
    H, hk, hd, page, T = 3, 1, 64, 32, 40
    pages = R.Pages([T], hk, page, hd, "f32", seed=111)
    raw = torch.randn((T, (H + 2) * hd + 3), generator=torch.Generator().manual_seed(1))
    f = _freqs(64)
    pos = np.arange(T) * 26001 + 12345            # up to a million
    for skew in (0, 1):
        buf = raw.cuda()
        view = buf.as_strided((T, H + 2, hd), (raw.shape[1], hd, 1), skew)
        x = R.f64(view)
        kv = pages.cuda(ms)
        out = ms.rope_append_paged(kv, view[:, :H], view[:, H:H + 1], view[:, H + 1:], R.starts([T]).cuda(), f.cuda(),
                                   positions=torch.tensor(pos, dtype=torch.int32).cuda(), out=view[:, :H])
        want = R.rotate(x[:, :H + 1], pos, f.numpy(), False, 1.0)
        assert np.all(np.abs(R.f64(out) - want[:, :H]) <= _rope_tol("f32", want[:, :H], x[:, :H], 1.0))
        assert np.array_equal(R.f64(view)[:, H:], x[:, H:])      # k and v are only read


def test_append_alone_and_many_rows():
    # q None: k and v alone; enough rows that a block takes several
    hk, hd, page, T = 1, 64, 256, 5200
    pages = R.Pages([0, 0], hk, page, hd, "f16", seed=121, extra=T)
    kv = pages.cuda(ms, lens=[T, 17])
    k = torch.randn((T + 17, hk, hd), device="cuda")
    v = torch.randn((T + 17, hk, hd), device="cuda")
    f = _freqs(64)
    assert ms.rope_append_paged(kv, None, k, v, R.starts([T, 17]).cuda(), f.cuda()) is None
    pos = np.concatenate([np.arange(T), np.arange(17)])
    x = R.f64(k)
    want = R.rotate(x, pos, f.numpy(), False, 1.0)
    gk, gv = R.f64(pages.dk), R.f64(pages.dv)
    tab = pages.table.numpy()
    b = np.repeat([0, 1], [T, 17])
    at = tab[b, pos // page]
    assert np.all(np.abs(gk[at, 0, pos % page] - want[:, 0]) <= _rope_tol("f16", want, x, 1.0)[:, 0])
    assert np.array_equal(gv[at, 0, pos % page], R.f64(v[:, 0].half()))


def test_append_flags_rows_without_a_place():
    pages = R.Pages([20, 20], 1, 16, 64, "f32", seed=131)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.randn((4, 1, 64), device="cuda")
    for lens, counts in (([33, 20], [1, 1]), ([20, 2], [1, 3]), ([20, -5], [1, 1])):
        kv = pages.cuda(ms, status, lens=lens)
        before = R.f64(pages.dk)
        ms.rope_append_paged(kv, None, x, x, R.starts(counts).cuda(), None)
        with pytest.raises(ms.MsError):
            ms.op_status(status)
        changed = ~((R.f64(pages.dk) == before) | (np.isnan(before) & np.isnan(R.f64(pages.dk))))
        assert changed.any(axis=(1, 3)).sum() <= sum(counts) - 1


# ---- eviction ----------------------------------------------------------------------------------

@pytest.mark.parametrize("kind,hd", [("f32", 64), ("f16", 64), ("bf16", 128), ("f32", 128)])
@pytest.mark.parametrize("keep,first,recent", [(16, 0, 0), (33, 4, 20), (64, 0, 64), (40, 40, 0), (1, 0, 0), (250, 1, 2), (700, 0, 5)])
@pytest.mark.parametrize("weights", ["spread", "tied", "odd"])
def test_evict(kind, hd, keep, first, recent, weights):
    lens, hk, page = [1, 0, 16, 33, 64, 65, 300, 251], 2, 16
    pages = R.Pages(lens, hk, page, hd, kind, seed=141, spare=2 + sum(-(-min(t, keep) // page) for t in lens))
    g = torch.Generator().manual_seed(keep)
    cap = pages.max_pages * page
    ldw = max(cap, keep) + 5
    w = torch.exp(3 * torch.randn((len(lens), hk, ldw), generator=g))
    if weights == "tied":
        w = torch.randint(0, 3, w.shape, generator=g).float() - 1      # -1, 0 and 1; -0 among the zeros
        w[..., ::7] *= -0.0
    if weights == "odd":
        r = torch.rand(w.shape, generator=g)
        w = torch.where(r < 0.1, torch.full_like(w, float("inf")), w)
        w = torch.where((r > 0.1) & (r < 0.2), torch.full_like(w, float("nan")), w)
        w = torch.where((r > 0.2) & (r < 0.3), torch.full_like(w, -float("inf")), w)
        w = torch.where((r > 0.3) & (r < 0.4), torch.full_like(w, 1e-42), w)
    dst = torch.full((len(lens), -(-keep // page)), 1 << 29, dtype=torch.int32)
    free = list(pages.free)
    for b, t in enumerate(lens):
        for j in range(-(-min(t, keep) // page)):
            dst[b, j] = free.pop()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = pages.cuda(ms, status)
    outs = []
    for in_place in (False, True):
        dw = w.cuda()
        kept, new, nl = ms.evict_paged(kv, dw, dst.cuda(), keep, first=first, recent=recent, weights_out=dw if in_place else None)
        ms.op_status(status)
        outs.append((kept.cpu().numpy(), new.cpu().numpy(), nl.cpu().numpy()))
    gk, gv = R.f64(pages.dk), R.f64(pages.dv)
    wn = w.numpy()
    for b, t in enumerate(lens):
        k, v = pages.rows("k", b), pages.rows("v", b)
        for h in range(hk):
            ids = R.evict(wn[b, h], t, keep, first, recent)
            m = len(ids)
            for kept, new, nl in outs:
                assert np.array_equal(kept[b, h, :m], ids) and np.all(kept[b, h, m:] == -1)
                assert np.array_equal(new[b, h, :m], wn[b, h, ids], equal_nan=True) and np.all(new[b, h, m:] == 0)
                assert nl[b] == m
            for j, i in enumerate(ids):
                p = int(dst[b, j // page])
                assert np.array_equal(gk[p, h, j % page], k[h, i]) and np.array_equal(gv[p, h, j % page], v[h, i])


def test_evict_long_rows_and_kept_pages():
    # several chunks of positions; the second sequence keeps all and keeps its pages
    lens, hk, page, hd, keep = [9001, 500], 1, 256, 64, 4100
    pages = R.Pages([0, 0], hk, page, hd, "f16", seed=151, extra=9001, spare=20)
    kv = pages.cuda(ms, lens=lens)
    pages.dk.normal_()
    pages.dv.normal_()
    before = pages.dk.clone()
    w = torch.rand((2, 1, kv.capacity), device="cuda")
    dst = torch.zeros((2, 17), dtype=torch.int32)
    dst[0, :17] = torch.tensor(pages.free[:17], dtype=torch.int32)
    dst[1, :2] = pages.table[1, :2]
    kept, new, nl = ms.evict_paged(kv, w, dst.cuda(), keep, recent=1000)
    wn = w.cpu().numpy()
    ids = R.evict(wn[0, 0], 9001, keep, 0, 1000)
    assert np.array_equal(kept.cpu().numpy()[0, 0], ids)
    assert np.array_equal(kept.cpu().numpy()[1, 0, :500], np.arange(500))
    assert nl.cpu().tolist() == [4100, 500]
    src = before[pages.table[0].long().cuda(), 0].reshape(-1, hd)[torch.from_numpy(ids).cuda()]
    assert torch.equal(pages.dk[dst[0].long().cuda(), 0].reshape(-1, hd)[:keep], src)
    assert torch.equal(pages.dk[dst[1, :2].long().cuda()], before[dst[1, :2].long().cuda()])


def test_evict_flags_bad_pages_and_lengths():
    pages = R.Pages([40, 40], 1, 16, 64, "f32", seed=161, spare=6)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dst = torch.tensor([[pages.free[0]], [pages.free[1]]], dtype=torch.int32)
    for what in ("dst", "src", "len"):
        kv = pages.cuda(ms, status, lens=[40, 4000] if what == "len" else None)
        d = dst.cuda()
        if what == "dst":
            d[1, 0] = -1
        if what == "src":
            pages.dtable[1] = pages.n_pages
        ms.evict_paged(kv, torch.rand((2, 1, kv.capacity), device="cuda"), d, 16)
        with pytest.raises(ms.MsError):
            ms.op_status(status)
        k = R.f64(pages.dk)
        assert np.all(np.isfinite(k[int(dst[0, 0])]))


# ---- verification of drafts ------------------------------------------------------------------

def _probs(rows, V, seed, sharp=3.0):
    g = torch.Generator().manual_seed(seed)
    return torch.softmax(torch.randn((rows, V), generator=g) * sharp, 1)


def _check_verify(target, draft, tokens, counts, ua, us, most):
    taken, said = R.verify(target.numpy(), None if draft is None else draft.numpy(), tokens.numpy(), counts, ua.numpy(), us.numpy())
    acc, out = ms.verify_draft(target.cuda(), None if draft is None else draft.cuda(), tokens.cuda(), R.starts(counts).cuda(),
                               most, ua.cuda(), us.cuda())
    assert acc.cpu().tolist() == taken
    for row, want in zip(out.cpu().tolist(), said):
        assert row == want + [-1] * (most + 1 - len(want))
    return taken


@pytest.mark.parametrize("V", [1, 2, 31, 1393, 4097, 32003, 100003])
@pytest.mark.parametrize("with_draft", [True, False])
def test_verify(V, with_draft):
    counts = [0, 1, 4, 8, 3, 8, 2, 5]
    n, B = sum(counts), len(counts)
    target = _probs(n + B, V, seed=V)
    g = torch.Generator().manual_seed(V + 1)
    own = torch.tensor([r + b for b, (a, c) in enumerate(zip(np.cumsum([0] + counts), counts)) for r in range(a, a + c)])
    draft = target[own] * torch.exp(0.5 * torch.randn((n, V), generator=g))
    draft = draft / draft.sum(1, keepdim=True)
    tokens = torch.multinomial(draft, 1, generator=g)[:, 0].to(torch.int32)
    ua, us = torch.rand(n, generator=g), torch.rand(B, generator=g)
    us[0], us[1] = 0.0, 1 - 2.0 ** -24
    taken = _check_verify(target, draft if with_draft else None, tokens, counts, ua, us, 8)
    if V > 1000 and with_draft:
        assert 0 < sum(taken) < n


def test_verify_extremes():
    V, counts = 500, [3, 3, 3, 3]
    target = _probs(16, V, seed=3)
    own = torch.tensor([0, 1, 2, 4, 5, 6, 8, 9, 10, 12, 13, 14])
    draft = target[own].clone()                     # equal distributions: every draft stays
    g = torch.Generator().manual_seed(9)
    tokens = torch.multinomial(draft, 1, generator=g)[:, 0].to(torch.int32)
    ua, us = torch.rand(12, generator=g), torch.rand(4, generator=g)
    assert _check_verify(target, draft, tokens, counts, ua, us, 3) == [3, 3, 3, 3]
    # a token the target never takes, refused where the two rows are the same: the draw falls back to p
    target[0, 7] = 0.0
    draft[0] = target[0]
    tokens[0] = 7
    assert _check_verify(target, draft, tokens, counts, ua, us, 3)[0] == 0
    # all weight on the last token; tokens without weight before and behind are never drawn
    target[4:8] = 0
    target[4:8, V - 1] = 1.0
    us[1] = 1 - 2.0 ** -24
    _check_verify(target, draft, tokens, counts, ua, us, 3)
    _check_verify(target, None, tokens, counts, ua, us, 3)


def test_verify_flags_bad_tokens_rows_and_empty_distributions():
    V = 300
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    target, draft = _probs(6, V, seed=4).cuda(), _probs(4, V, seed=5).cuda()
    tok = torch.tensor([1, 2, 3, 4], dtype=torch.int32)
    u = torch.full((4,), 0.5, device="cuda")
    for what, code in (("token", ms.MS_ERR_TOKEN_RANGE), ("empty", ms.MS_ERR_TOKEN_RANGE), ("rows", ms.MS_ERR_SHAPE)):
        t2, target2, st = tok.clone(), target.clone(), R.starts([2, 2])
        if what == "token":
            t2[0] = V
        if what == "empty":
            target2[0] = 0.0
        if what == "rows":
            st[1] = 5
        acc, out = ms.verify_draft(target2, draft, t2.cuda(), st.cuda(), 2, u, u[:2].contiguous(), status)
        with pytest.raises(ms.MsError) as e:
            ms.op_status(status)
        assert e.value.status == code
        assert acc[0].item() == 0
        if what == "empty":
            assert out[0, 0].item() == -1
        if what == "rows":
            assert out.cpu().tolist() == [[-1] * 3] * 2
