"""The paged-cache operators together, as a server runs them: append, attend, verify, cut back, go on; eagerly and in a
captured graph.  Each step is held against the 64-bit restatements on what the cache then holds.  Tolerances are those
of test_paged_gpu.py."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_ref as R
from test_paged_gpu import _attn_tol, _check_attn, _freqs, _probs, _rope_tol

pytestmark = pytest.mark.gpu
ms = pytest.importorskip("decoder_only_transformer_int4_b200")


class Server:
    """Three sequences over one pool; the host keeps lengths, true positions and free pages."""

    def __init__(self, kq, kkv, hd, hk, H, page, graph, seed):
        self.kq, self.kkv, self.hd, self.hk, self.H, self.page = kq, kkv, hd, hk, H, page
        self.rng = np.random.default_rng(seed)
        self.g = torch.Generator().manual_seed(seed)
        self.pages = R.Pages([0, 0, 0], hk, page, hd, kkv, seed, spare=40, extra=6 * page)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.kv = self.pages.cuda(ms, self.status)
        self.lens, self.pos = [0, 0, 0], [0, 0, 0]
        self.weights = torch.zeros((3, hk, self.kv.capacity), device="cuda")
        self.freq = _freqs(hd)
        self.most, self.V = 5, 700
        rows = 3 * self.most
        t = R.TYPES[kq]
        self.b = dict(x=torch.zeros((rows, H + 2 * hk, hd), dtype=t, device="cuda"), out=torch.zeros((rows, H, hd), dtype=t, device="cuda"),
                      attn=torch.zeros((rows, H, hd), dtype=t, device="cuda"), start=torch.zeros(4, dtype=torch.int32, device="cuda"),
                      pos=torch.zeros(rows, dtype=torch.int32, device="cuda"), freq=self.freq.cuda(),
                      target=torch.zeros((rows, self.V), device="cuda"), draft=torch.zeros((rows - 3, self.V), device="cuda"),
                      tok=torch.zeros(rows - 3, dtype=torch.int32, device="cuda"), dstart=torch.zeros(4, dtype=torch.int32, device="cuda"),
                      ua=torch.zeros(rows - 3, device="cuda"), us=torch.zeros(3, device="cuda"))
        self.graph = None
        if graph:
            self.calls()                      # before the capture: attributes are set, nothing else is kept
            torch.cuda.synchronize()
            self.weights.zero_()
            self.status.zero_()               # probabilities of zero were flagged
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.calls()

    def calls(self):
        b, H, hk = self.b, self.H, self.hk
        ms.rope_append_paged(self.kv, b["x"][:, :H], b["x"][:, H:H + hk], b["x"][:, H + hk:], b["start"], b["freq"], positions=b["pos"], out=b["out"])
        ms.attn_paged(self.kv, b["out"], b["start"], self.most, weights=self.weights, out=b["attn"])
        self.said = ms.verify_draft(b["target"], b["draft"], b["tok"], b["dstart"], self.most - 1, b["ua"], b["us"], self.status)

    def step(self, counts):
        """One step of counts[b] rows (drafts after the first) of each sequence; the refused ones leave the cache again."""
        b, H, hk, page = self.b, self.H, self.hk, self.page
        rows, n = sum(counts), sum(max(c - 1, 0) for c in counts)
        for i, c in enumerate(counts):
            self.lens[i] += c
        b["x"].copy_(torch.randn(b["x"].shape, generator=self.g).to(b["x"].dtype))
        b["out"].fill_(7.0)
        b["attn"].fill_(7.0)
        b["start"].copy_(R.starts(counts))
        at = np.concatenate([np.arange(p, p + c) for p, c in zip(self.pos, counts)] + [np.zeros(15 - rows)])
        b["pos"].copy_(torch.tensor(at, dtype=torch.int32))
        drafts = [max(c - 1, 0) for c in counts]
        b["dstart"].copy_(R.starts(drafts))
        target, ua, us = _probs(15, self.V, int(self.rng.integers(1 << 30))), torch.rand(12, generator=self.g), torch.rand(3, generator=self.g)
        own = [r + i for i, (a, c) in enumerate(zip(np.cumsum([0] + drafts), drafts)) for r in range(a, a + c)]
        draft = _probs(12, self.V, int(self.rng.integers(1 << 30)))
        draft[:n] = target[own] * torch.exp(0.4 * torch.randn((n, self.V), generator=self.g))
        draft /= draft.sum(1, keepdim=True)
        tok = torch.multinomial(draft, 1, generator=self.g)[:, 0].to(torch.int32)
        for name, v in (("target", target), ("draft", draft), ("tok", tok), ("ua", ua), ("us", us)):
            b[name].copy_(v)
        self.pages.dlens.copy_(torch.tensor(self.lens, dtype=torch.int32))
        before = R.f64(self.weights)
        if self.graph is None:
            self.calls()
        else:
            self.graph.replay()
        ms.op_status(self.status)

        # rotary and append
        P = self.pages
        P.k, P.v, P.table, P.lens = P.dk.cpu(), P.dv.cpu(), P.dtable.cpu(), list(self.lens)
        x = R.f64(b["x"])[:rows]
        want = R.rotate(x[:, :H + hk], at[:rows], self.freq.numpy(), False, 1.0)
        assert np.all(np.abs(R.f64(b["out"])[:rows] - want[:, :H]) <= _rope_tol(self.kq, want[:, :H], x[:, :H], 1.0))
        assert np.all(R.f64(b["out"])[rows:] == 7.0) and np.all(R.f64(b["attn"])[rows:] == 7.0)
        r = 0
        for i, c in enumerate(counts):
            for j in range(c):
                t = self.lens[i] - c + j
                p = int(P.table[i, t // page])
                tol = _rope_tol(self.kkv, want[r, H:], x[r, H:H + hk], 1.0)
                assert np.all(np.abs(R.f64(P.k[p, :, t % page]) - want[r, H:]) <= tol)
                assert np.array_equal(R.f64(P.v[p, :, t % page]), R.f64(b["x"][r, H + hk:].to(R.TYPES[self.kkv])))
                r += 1
        # attention over what the cache holds
        scale = self.hd ** -0.5
        ref, A, spread, rw = R.attention(P, b["out"][:rows], counts, scale)
        T = np.repeat(np.array(self.lens), counts)[:, None]
        assert np.all(np.abs(R.f64(b["attn"])[:rows] - ref) <= _attn_tol(self.kq, self.kkv, self.hd, T, ref, A, spread))
        after = R.f64(self.weights)
        for i, t in enumerate(self.lens):
            assert np.array_equal(after[i, :, t:], before[i, :, t:])
            sp = spread[sum(counts[:i]):sum(counts[:i + 1])].max(initial=0.0)
            rel = 2 * (self.hd + 17) * 2.0 ** -23 * sp + (8 + 2 * t + 64) * 2.0 ** -23
            assert np.all(np.abs(after[i, :, :t] - before[i, :, :t] - rw[i]) <= rel * rw[i] + 2.0 ** -23 * (before[i, :, :t] + rw[i]))
        # drafts
        taken, said = R.verify(target.numpy(), draft.numpy(), tok.numpy(), drafts, ua.numpy(), us.numpy())
        acc, out = self.said
        assert acc.cpu().tolist() == taken
        for row, w in zip(out.cpu().tolist(), said):
            assert row == w + [-1] * (self.most - len(w))
        for i, c in enumerate(counts):
            refused = drafts[i] - taken[i]
            self.lens[i] -= refused
            self.pos[i] += c - refused
            self.weights[i, :, self.lens[i]:] = 0
        return taken

    def cut(self, keep, first, recent):
        P, page = self.pages, self.page
        self.pages.dlens.copy_(torch.tensor(self.lens, dtype=torch.int32))
        dst = P.dtable.cpu().clone()
        old = []
        for i, t in enumerate(self.lens):
            if t > keep:
                for j in range(-(-keep // page)):
                    old.append(int(dst[i, j]))
                    dst[i, j] = P.free.pop(0)
        w = R.f64(self.weights)
        P.k, P.v, P.table, P.lens = P.dk.cpu(), P.dv.cpu(), P.dtable.cpu(), list(self.lens)
        want = [(P.rows("k", i), P.rows("v", i)) for i in range(3)]
        ddst = dst.cuda()
        kept, new, lens = ms.evict_paged(self.kv, self.weights, ddst, keep, first=first, recent=recent, weights_out=self.weights)
        ms.op_status(self.status)
        self.pages.dtable.copy_(ddst)
        P.k, P.v, P.table = P.dk.cpu(), P.dv.cpu(), P.dtable.cpu()
        for i, t in enumerate(self.lens):
            P.lens[i] = min(t, keep)
            k, v = P.rows("k", i), P.rows("v", i)
            for h in range(self.hk):
                ids = R.evict(w[i, h], t, keep, first, recent)
                assert np.array_equal(kept[i, h, :len(ids)].cpu().numpy(), ids)
                assert np.array_equal(R.f64(new)[i, h, :len(ids)], w[i, h, ids]) and np.all(R.f64(new)[i, h, len(ids):] == 0)
                assert np.array_equal(k[h], want[i][0][h][ids]) and np.array_equal(v[h], want[i][1][h][ids])
        assert lens.cpu().tolist() == P.lens
        self.lens = list(P.lens)
        P.free += old


@pytest.mark.parametrize("kq,kkv", R.PAIRS)
@pytest.mark.parametrize("hd,hk,H,page", [(64, 2, 8, 16), (128, 1, 7, 32)])
@pytest.mark.parametrize("graph", [False, True])
def test_a_run_of_the_operators(kq, kkv, hd, hk, H, page, graph):
    s = Server(kq, kkv, hd, hk, H, page, graph, seed=171)
    s.step([5, 1, 0])
    total = 0
    for i in range(7):
        total += sum(s.step([5, 1 + i % 4, 3]))
    assert 0 < total
    s.cut(keep=11, first=1, recent=4)
    assert max(s.lens) == 11 and max(s.pos) > 11      # cache index and position differ from here on
    for i in range(3):
        s.step([1, 5, i])
    s.cut(keep=6, first=0, recent=6)
    s.step([5, 5, 5])


# ---- attention where the work is cut in many ways ----------------------------------------------

@pytest.mark.parametrize("kq,kkv", R.PAIRS)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("group,counts", [(8, [5, 2, 4, 0, 1, 7]), (3, [1, 1, 1, 1, 1, 1]), (5, [4, 3, 0, 2, 2, 6]), (24, [1, 0, 3, 2, 1, 1])])
def test_attention_runs_over_units_of_all_lengths(kq, kkv, hd, group, counts):
    # a table of more than 16 tiles: runs of tiles, not clusters; one to four row tiles, one to three passes
    _check_attn(kq, kkv, hd, 1, group, 32, [1090, 0, 3, 64, 400, 129], counts, seed=181 + group, weights=True)


@pytest.mark.parametrize("kq,kkv", R.PAIRS)
@pytest.mark.parametrize("group,most", [(8, 4), (16, 3), (1, 33)])
def test_attention_in_clusters_with_several_row_tiles(kq, kkv, group, most):
    lens = [300, 0, 15, 64, 257]
    counts = [most, 1, most, 0, 2]
    _check_attn(kq, kkv, 64, 2, group, 16, lens, counts, seed=191 + group, weights=True, most=most)


def test_attention_of_many_sequences():
    lens = [(37 * i) % 90 for i in range(300)]
    _check_attn("f16", "f16", 64, 1, 2, 16, lens, [i % 3 for i in range(300)], seed=201, weights=True)


@pytest.mark.parametrize("kq,kkv", R.PAIRS)
def test_attention_scores_that_fall_and_rise(kq, kkv):
    # the running reference: scores that grow along the sequence, in small steps and in jumps past any slack
    T = 700
    for growth in (0.02, 0.5):
        pages = R.Pages([T], 1, 16, 64, kkv, seed=211)
        for i in range(T):
            p = int(pages.table[0, i // 16])
            pages.k[p, 0, i % 16] = torch.full((64,), 0.0)
            pages.k[p, 0, i % 16, 0] = growth * (i if i % 50 else i + 40)
        q = torch.zeros((1, 4, 64))
        q[..., 0] = torch.tensor([1.0, -1.0, 0.25, 0.0])
        q = q.to(R.TYPES[kq])
        got = R.f64(ms.attn_paged(pages.cuda(ms), q.cuda(), R.starts([1]).cuda(), 1, scale=1.0))
        ref, A, spread, _ = R.attention(pages, q, [1], 1.0)
        assert np.all(np.abs(got - ref) <= _attn_tol(kq, kkv, 64, np.array([[T]]), ref, A, spread))


def test_attention_calls_in_a_row_share_a_workspace():
    # one stream: the second call's kernels may begin while the first one's end, but not touch the workspace before
    lens = [1500, 40, 900]
    pages = R.Pages(lens, 2, 64, 64, "f16", seed=221)
    kv = pages.cuda(ms)
    st = R.starts([1, 1, 1]).cuda()
    ws = torch.empty(ms.attn_paged_workspace(kv, torch.float16, 8, 1, True), dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(3)
    qs = [torch.randn((3, 8, 64), generator=g).half() for _ in range(20)]
    w = torch.zeros((3, 2, kv.capacity), device="cuda")
    dq = [q.cuda() for q in qs]
    torch.cuda.synchronize()
    outs = [ms.attn_paged(kv, q, st, 1, weights=w, workspace=ws) for q in dq]
    want, rel = np.zeros(w.shape), 0.0
    for q, o in zip(qs, outs):
        ref, A, spread, rw = R.attention(pages, q, [1, 1, 1], 0.125)
        assert np.all(np.abs(R.f64(o) - ref) <= _attn_tol("f16", "f16", 64, np.array(lens)[:, None], ref, A, spread))
        rel = max(rel, 2 * (64 + 17) * 2.0 ** -23 * spread.max())
        for b, t in enumerate(lens):
            want[b, :, :t] += rw[b]
    # the probabilities' relative error as in test_paged_gpu.py, and one rounding for each of 20 additions
    assert np.all(np.abs(R.f64(w) - want) <= (rel + (8 + 2 * 1500 + 4) * 2.0 ** -23 + 20 * 2.0 ** -24) * want)


# ---- eviction where a sequence is shared by many CTAs ---------------------------------------------

@pytest.mark.parametrize("T,keep,first,recent", [(9001, 4100, 3, 500), (9001, 9000, 0, 0), (20000, 37, 0, 5), (100003, 50001, 10, 1000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_over_a_cluster(T, keep, first, recent, in_place):
    hk, page, hd = 2, 256, 64
    need, more = -(-T // page), -(-keep // page)
    g = torch.Generator(device="cuda").manual_seed(T)
    k = torch.randn((need + more, hk, page, hd), generator=g, device="cuda").half()
    v = torch.randn((need + more, hk, page, hd), generator=g, device="cuda").half()
    order = torch.randperm(need + more, generator=g, device="cuda").to(torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = ms.PagedKV(k, v, order[:need].reshape(1, -1).contiguous(), torch.tensor([T], dtype=torch.int32, device="cuda"), status)
    w = torch.randint(0, 1000, (1, hk, kv.capacity), generator=g, device="cuda").float()   # many ties
    before, k0, v0 = w.cpu().numpy(), k.clone(), v.clone()
    dst = order[need:].reshape(1, -1).contiguous()
    kept, new, lens = ms.evict_paged(kv, w, dst, keep, first=first, recent=recent, weights_out=w if in_place else None)
    ms.op_status(status)
    assert lens.cpu().tolist() == [keep]
    src, to = order[:need].long(), order[need:].long()
    for h in range(hk):
        ids = R.evict(before[0, h], T, keep, first, recent)
        assert np.array_equal(kept[0, h].cpu().numpy(), ids)
        assert np.array_equal(new[0, h, :keep].cpu().numpy(), before[0, h, ids]) and not new[0, h, keep:].any()
        at = torch.from_numpy(ids).cuda()
        for x, x0 in ((k, k0), (v, v0)):
            assert torch.equal(x[to, h].reshape(-1, hd)[:keep], x0[src, h].reshape(-1, hd)[at])
    assert torch.equal(k[src], k0[src]) and torch.equal(v[src], v0[src])


def test_evict_keeps_more_than_the_tables_hold():
    # no sequence reaches keep: narrower tables and weights than keep are enough
    lens, hk, page, keep = [50, 3, 0, 33], 2, 16, 200
    pages = R.Pages(lens, hk, page, 64, "bf16", seed=281, spare=20)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = pages.cuda(ms, status)
    w = torch.rand((4, hk, kv.capacity), device="cuda")
    assert kv.capacity < keep
    dst = torch.full((4, 4), 1 << 29, dtype=torch.int32)
    for b, t in enumerate(lens):
        for j in range(-(-t // page)):
            dst[b, j] = pages.free.pop()
    for narrow in (4, 3):
        kept, new, nl = ms.evict_paged(kv, w, dst[:, :narrow].contiguous().cuda(), keep, first=3, recent=100)
        if narrow == 4:
            ms.op_status(status)
        else:                                  # the first sequence's last two rows have no page: left out and flagged
            with pytest.raises(ms.MsError):
                ms.op_status(status)
        assert nl.cpu().tolist() == lens
        k = R.f64(pages.dk)
        for b, t in enumerate(lens):
            src = pages.rows("k", b)
            assert np.array_equal(kept[b, 0].cpu().numpy(), list(range(t)) + [-1] * (keep - t))
            assert torch.equal(new[b, :, :t], w[b, :, :t]) and not new[b, :, t:].any()
            for j in range(min(t, narrow * page)):
                assert np.array_equal(k[int(dst[b, j // page]), :, j % page], src[:, j])


# ---- the handle, other streams -------------------------------------------------------------------------

def test_the_cache_keeps_its_tensors_and_is_read_only():
    pages = R.Pages([40], 1, 16, 64, "f32", seed=231)
    q = torch.randn((1, 2, 64), generator=torch.Generator().manual_seed(6))
    kv = pages.cuda(ms)
    ref, A, spread, _ = R.attention(pages, q, [1], 0.125)
    with pytest.raises(AttributeError):
        kv.lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    del pages.dk, pages.dv, pages.dtable, pages.dlens
    junk = [torch.full((1 << 18,), 1e30, device="cuda") for _ in range(8)]
    got = R.f64(ms.attn_paged(kv, q.cuda(), R.starts([1]).cuda(), 1))
    assert np.all(np.abs(got - ref) <= _attn_tol("f32", "f32", 64, np.array([[40]]), ref, A, spread))
    assert (kv.n_kv_heads, kv.head_dim, kv.capacity, kv.batch) == (1, 64, 48, 1) and len(junk) == 8


def test_calls_run_on_the_current_stream():
    lens = [1500, 300]
    pages = R.Pages(lens, 1, 64, 64, "f16", seed=241)
    q = torch.randn((2, 4, 64), generator=torch.Generator().manual_seed(8))
    ref, A, spread, _ = R.attention(pages, q, [1, 1], 0.125)
    kv, st = pages.cuda(ms), R.starts([1, 1]).cuda()
    streams = [torch.cuda.Stream() for _ in range(3)]
    dq = [q.cuda() for _ in streams]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for s, x in zip(streams, dq):
            with torch.cuda.stream(s):
                outs.append(ms.attn_paged(kv, x, st, 1))       # each call a workspace of its own
    torch.cuda.synchronize()
    tol = _attn_tol("f32", "f16", 64, np.array(lens)[:, None], ref, A, spread)
    for o in outs:
        assert np.all(np.abs(R.f64(o) - ref) <= tol)


def test_python_calls_refuse_wrong_tensors():
    pages = R.Pages([40, 3], 2, 16, 64, "f16", seed=251, spare=6)
    kv = pages.cuda(ms)
    q, st = torch.zeros((2, 4, 64), dtype=torch.float16, device="cuda"), R.starts([1, 1]).cuda()
    w = torch.zeros((2, 2, kv.capacity), device="cuda")
    ok = lambda **c: ms.attn_paged(**{**dict(kv=kv, q=q, row_start=st, max_rows=1, weights=w), **c})  # noqa: E731
    ok()
    for bad in (dict(q=q[:, :, :32]), dict(q=q[0]), dict(q=q.transpose(0, 1)), dict(q=q.cpu()), dict(q=q.double()), dict(row_start=st[:2]),
                dict(row_start=st.long()), dict(row_start=st.cpu()), dict(weights=w[:1]), dict(weights=w.half()), dict(weights=w[..., ::2]),
                dict(out=q[:1]), dict(out=q.float()), dict(workspace=torch.empty(10, device="cuda"))):
        with pytest.raises(ValueError):
            ok(**bad)
    for bad, code in ((dict(q=q.bfloat16()), ms.MS_ERR_UNSUPPORTED), (dict(max_rows=0), ms.MS_ERR_SHAPE), (dict(q=q[:, :3].contiguous()), ms.MS_ERR_SHAPE),
                      (dict(weights=w[..., :16].contiguous()), ms.MS_ERR_SHAPE), (dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda")), ms.MS_ERR_SHAPE),
                      (dict(scale=float("inf")), ms.MS_ERR_INVALID_ARG)):
        with pytest.raises(ms.MsError) as e:
            ok(**bad)
        assert e.value.status == code
    k = torch.zeros((2, 2, 64), dtype=torch.float16, device="cuda")
    f = _freqs(64).cuda()
    for bad in (dict(k=k[:1]), dict(v=k[:1]), dict(inv_freq=f.float()), dict(inv_freq=f[None]), dict(positions=st), dict(q=None, out=q), dict(q=q[:1])):
        with pytest.raises(ValueError):
            ms.rope_append_paged(**{**dict(kv=kv, q=q, k=k, v=k, row_start=st, inv_freq=f), **bad})
    for bad in (dict(weights=w[0]), dict(dst_table=st), dict(weights_out=w.half())):
        with pytest.raises(ValueError):
            ms.evict_paged(**{**dict(kv=kv, weights=w, dst_table=st[:2].reshape(2, 1), keep=4), **bad})
    for bad in (pages.dtable[0], pages.dtable.long(), pages.dtable.cpu()):
        with pytest.raises(ValueError):
            ms.PagedKV(pages.dk, pages.dv, bad, pages.dlens)
    with pytest.raises(ValueError):
        ms.PagedKV(pages.dk, pages.dv[:1], pages.dtable, pages.dlens)
    with pytest.raises(ValueError):
        ms.PagedKV(pages.dk.transpose(1, 2), pages.dv.transpose(1, 2), pages.dtable, pages.dlens)
    with pytest.raises(ValueError):
        ms.PagedKV(pages.dk, pages.dv, pages.dtable, pages.dlens[:1])


def test_verify_refuses_random_numbers_outside_their_range():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    target = _probs(2, 300, seed=5).cuda()
    none, empty = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(0, device="cuda")
    for u in (1.0, -0.1, float("nan"), float("inf")):
        acc, out = ms.verify_draft(target, None, none, R.starts([0, 0]).cuda(), 0, empty, torch.tensor([0.5, u], device="cuda"), status)
        with pytest.raises(ms.MsError) as e:
            ms.op_status(status)
        assert e.value.status == ms.MS_ERR_TOKEN_RANGE
        assert out[0, 0].item() >= 0 and out[1, 0].item() == -1 and acc.cpu().tolist() == [0, 0]


@pytest.mark.parametrize("kq,kkv", R.PAIRS)
@pytest.mark.parametrize("lens", [[1500, 64, 0, 700], [300, 64, 0, 70]])
def test_attention_in_place_of_its_queries(kq, kkv, lens):
    pages = R.Pages(lens, 2, 16, 64, kkv, seed=261)
    counts = [2, 1, 1, 3]
    q = torch.randn((7, 8, 64), generator=torch.Generator().manual_seed(12)).to(R.TYPES[kq])
    x = q.cuda()
    assert ms.attn_paged(pages.cuda(ms), x, R.starts(counts).cuda(), 3, out=x) is x
    ref, A, spread, _ = R.attention(pages, q, counts, 0.125)
    T = np.repeat(np.array(lens), counts)[:, None]
    assert np.all(np.abs(R.f64(x) - ref) <= _attn_tol(kq, kkv, 64, T, ref, A, spread))


def test_rope_turns_back_at_negative_positions():
    pages = R.Pages([6], 2, 16, 64, "f32", seed=271)
    x = torch.randn((6, 2, 64), generator=torch.Generator().manual_seed(4))
    f = _freqs(64)
    pos = np.array([-1, -17, -1000, -65537, 0, -(2 ** 20)])
    out = ms.rope_append_paged(pages.cuda(ms), x.cuda(), x.cuda(), x.cuda(), R.starts([6]).cuda(), f.cuda(),
                               positions=torch.tensor(pos, dtype=torch.int32).cuda())
    want = R.rotate(R.f64(x), pos, f.numpy(), False, 1.0)
    assert np.all(np.abs(R.f64(out) - want) <= _rope_tol("f32", want, R.f64(x), 1.0))


FIRST = """
import numpy as np, torch
import paged_ref as R
import decoder_only_transformer_int4_b200 as ms
pages = R.Pages([1300, 40], 1, 16, 64, "f16", seed=5, spare=60)
kv = pages.cuda(ms)
q = torch.randn((2, 4, 64), generator=torch.Generator().manual_seed(1)).half()
dq, st = q.cuda(), R.starts([1, 1]).cuda()
w = torch.zeros((2, 1, kv.capacity), device="cuda")
dst = torch.tensor(pages.free[:4], dtype=torch.int32).reshape(2, 2).cuda()
p = torch.softmax(torch.randn((2, 50), generator=torch.Generator().manual_seed(2)), 1).cuda()
none, u = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.rand(2, device="cuda")
k, f, empty = torch.zeros((2, 1, 64), device="cuda").half(), torch.ones(32, dtype=torch.float64, device="cuda"), torch.zeros(0, device="cuda")
ref, _, _, rw = R.attention(pages, q, [1, 1], 0.125)
ZERO = R.starts([0, 0]).cuda()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):                     # nothing of the library has run yet
    out = ms.attn_paged(kv, dq, st, 1, weights=w)
    kept, new, lens = ms.evict_paged(kv, w, dst, 32)
    acc, tok = ms.verify_draft(p, None, none, ZERO, 0, empty, u)
    ms.rope_append_paged(kv, None, k, k, ZERO, f)
graph.replay()
torch.cuda.synchronize()
assert np.abs(R.f64(out) - ref).max() < 2e-3, np.abs(R.f64(out) - ref).max()
assert lens.cpu().tolist() == [32, 32] and acc.cpu().tolist() == [0, 0]
assert np.abs(R.f64(w)[0, :, :1300] - rw[0]).max() < 1e-4
print("done")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(here), here]))
    r = subprocess.run([sys.executable, "-c", FIRST], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("kq,kkv", R.PAIRS)
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_runs_of_many_tiles_over_several_units(kq, kkv, hd):
    # every CTA goes through more than 16 tiles (its descriptors are looked up in parts) and from unit to unit on the way
    g = torch.Generator(device="cuda").manual_seed(291)
    lens = [7000 + (977 * i) % 1300 for i in range(80)]
    group, page, scale = 2, 64, hd ** -0.5
    need = [-(-t // page) for t in lens]
    order = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((80, max(need)), dtype=torch.int32, device="cuda")
    for b, (n, o) in enumerate(zip(need, np.cumsum([0] + need))):
        table[b, :n] = order[o:o + n]
    k = torch.randn((sum(need), 1, page, hd), generator=g, device="cuda").to(R.TYPES[kkv])
    v = torch.randn((sum(need), 1, page, hd), generator=g, device="cuda").to(R.TYPES[kkv])
    q = torch.randn((80, group, hd), generator=g, device="cuda").to(R.TYPES[kq])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = ms.PagedKV(k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), status)
    out = R.f64(ms.attn_paged(kv, q, R.starts([1] * 80).cuda(), 1))
    ms.op_status(status)
    for b, t in enumerate(lens):
        kb = k[table[b, :need[b]].long(), 0].reshape(-1, hd)[:t].double()
        vb = v[table[b, :need[b]].long(), 0].reshape(-1, hd)[:t].double()
        p = torch.softmax((q[b].double() @ kb.T) * scale, 1)
        spread = (scale * (q[b].double().abs() @ kb.abs().T)).amax(1)
        ref, A = R.f64(p @ vb), R.f64(p @ vb.abs())
        tol = _attn_tol(kq, kkv, hd, np.full(group, t), ref, A, R.f64(spread))
        assert np.all(np.abs(out[b] - ref) <= tol), b


def test_offsets_past_32_bits():
    # four pages 2^31 elements and more apart, in one allocation of 13 GB; rows of probabilities as far apart
    hk, page, hd, T = 2, 64, 64, 150
    size, stride = hk * page * hd, 2 ** 31 + 64
    flat = torch.empty(3 * stride + 2 * size, dtype=torch.float16, device="cuda")
    k = flat.as_strided((4, hk, page, hd), (stride, page * hd, hd, 1), 0)
    v = flat.as_strided((4, hk, page, hd), (stride, page * hd, hd, 1), size)
    for x in (k, v):
        for i in range(4):
            x[i].fill_(float("nan"))
    pages = R.Pages([T], hk, page, hd, "f16", seed=301)
    pages.table = torch.tensor([[3, 0, 2]], dtype=torch.int32)
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = ms.PagedKV(k, v, pages.table.cuda(), lens, status)
    g = torch.Generator().manual_seed(302)
    x, f = torch.randn((T, 4 + 2 * hk, hd), generator=g).half(), _freqs(hd)
    d = x.cuda()
    q = ms.rope_append_paged(kv, d[:, :4], d[:, 4:4 + hk], d[:, 4 + hk:], R.starts([T]).cuda(), f.cuda())
    want = R.rotate(R.f64(x[:, :4 + hk]), np.arange(T), f.numpy(), False, 1.0)
    for i in range(T):
        got = R.f64(k[int(pages.table[0, i // page]), :, i % page])
        assert np.all(np.abs(got - want[i, 4:]) <= _rope_tol("f16", want[i, 4:], R.f64(x[i, 4:4 + hk]), 1.0))
    pages.k, pages.v, pages.lens = k.cpu(), v.cpu(), [T]
    w = torch.zeros((1, hk, kv.capacity), device="cuda")
    out = ms.attn_paged(kv, q[-2:].contiguous(), R.starts([2]).cuda(), 2, weights=w)
    ref, A, spread, _ = R.attention(pages, q[-2:], [2], hd ** -0.5)
    assert np.all(np.abs(R.f64(out) - ref) <= _attn_tol("f16", "f16", hd, np.array([[T]]), ref, A, spread))
    kept, _, _ = ms.evict_paged(kv, w, torch.tensor([[1]], dtype=torch.int32, device="cuda"), 50, first=2, recent=20)
    ms.op_status(status)
    rows = [pages.rows("k", 0), pages.rows("v", 0)]
    for h in range(hk):
        ids = kept[0, h].cpu().numpy()
        assert np.array_equal(R.f64(k[1, h, :50]), rows[0][h, ids]) and np.array_equal(R.f64(v[1, h, :50]), rows[1][h, ids])
    V = 5000
    target = flat.view(torch.float32)[:2 ** 31 + 8 + V].as_strided((2, V), (2 ** 31 + 8, 1), 0)
    p = _probs(2, V, seed=303)
    target.copy_(p)
    u = torch.tensor([0.3], device="cuda")
    tok = torch.tensor([int(p[0].argmax())], dtype=torch.int32)
    for ua in (0.0, 1 - 2.0 ** -24):
        acc, said = ms.verify_draft(target, None, tok.cuda(), R.starts([1]).cuda(), 1, torch.tensor([ua], device="cuda"), u)
        taken, words = R.verify(p.numpy(), None, tok.numpy(), [1], np.array([ua]), u.cpu().numpy())
        assert acc.cpu().tolist() == taken and said.cpu().tolist()[0] == words[0] + [-1] * (2 - len(words[0]))
