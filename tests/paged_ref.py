"""Plain 64-bit restatements of the paged-cache operators, and small caches to try them on (numpy and torch on
the CPU; nothing of the library)."""
import numpy as np
import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
PAIRS = [("f32", "f32"), ("f32", "f16"), ("f16", "f16"), ("bf16", "bf16")]


def half_step(kind):
    """Largest relative error of one rounding to the type."""
    return torch.finfo(TYPES[kind]).eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


class Pages:
    """A cache of random rows for the given lengths.  Every place that holds no position is NaN; the table's unused
    entries name no page."""

    def __init__(self, lens, hk, page, hd, kind, seed, spare=2, extra=0, gap=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hk, self.page, self.hd, self.kind = list(lens), hk, page, hd, kind
        need = [-(-(t + extra) // page) for t in lens]
        self.n_pages = sum(need) + spare
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.max_pages = max(1, max(need))
        self.table = torch.full((len(lens), self.max_pages), 1 << 29, dtype=torch.int32)
        for b, n in enumerate(need):
            for j in range(n):
                self.table[b, j] = order.pop()
        self.free = order
        shape = (self.n_pages, hk, page, hd)
        self.k = torch.full(shape, float("nan")).to(TYPES[kind])
        self.v = torch.full(shape, float("nan")).to(TYPES[kind])
        for b, t in enumerate(lens):
            for i in range(t):
                p = int(self.table[b, i // page])
                self.k[p, :, i % page] = torch.randn((hk, hd), generator=g).to(TYPES[kind])
                self.v[p, :, i % page] = torch.randn((hk, hd), generator=g).to(TYPES[kind])

    def rows(self, which, b, T=None):
        """[hk, T, hd] of sequence b, float64."""
        x = self.k if which == "k" else self.v
        T = self.lens[b] if T is None else T
        out = np.zeros((self.hk, T, self.hd))
        for i in range(T):
            out[:, i] = f64(x[int(self.table[b, i // self.page]), :, i % self.page])
        return out

    def cuda(self, ms, status=None, lens=None):
        self.dk, self.dv = self.k.cuda(), self.v.cuda()
        self.dtable = self.table.cuda()
        self.dlens = torch.tensor(self.lens if lens is None else lens, dtype=torch.int32).cuda()
        return ms.PagedKV(self.dk, self.dv, self.dtable, self.dlens, status)


def starts(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)


def attention(pages, q, counts, scale):
    """(out [rows, H, hd], its error scale, probabilities summed per position [b][hk][T], theirs) in float64.

    The error scale A = sum_t p_t |v_t| multiplies the relative error of the probabilities, of the sums and of the
    operands; `spread` is the largest sum of |q_d k_d| a row's scores are made of."""
    q = f64(q)
    H = q.shape[1]
    g = H // pages.hk
    out, A = np.zeros_like(q), np.zeros_like(q)
    spread = np.zeros(q.shape[:2])
    weights = [np.zeros((pages.hk, t)) for t in pages.lens]
    r = 0
    for b, (T, n) in enumerate(zip(pages.lens, counts)):
        k, v = pages.rows("k", b), pages.rows("v", b)
        for i in range(n):
            lim = T - n + i + 1
            for h in range(H):
                if lim <= 0:
                    continue
                kh, vh = k[h // g, :lim], v[h // g, :lim]
                s = scale * (kh @ q[r, h])
                spread[r, h] = abs(scale) * (np.abs(kh) @ np.abs(q[r, h])).max()
                p = np.exp(s - s.max())
                p /= p.sum()
                out[r, h] = p @ vh
                A[r, h] = p @ np.abs(vh)
                weights[b][h // g, :lim] += p
            r += 1
    return out, A, spread, weights


def rotate(x, pos, inv_freq, interleaved, mscale):
    """x [rows, heads, hd] float64 turned by its rows' positions."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    ang = np.asarray(pos, np.longdouble)[:, None] * np.asarray(inv_freq, np.longdouble)
    z = (np.cos(ang) + 0j).astype(np.complex128)
    z = (np.cos(ang).astype(np.float64) + 1j * np.sin(ang).astype(np.float64)) * mscale
    i0 = np.arange(half) * 2 if interleaved else np.arange(half)
    i1 = i0 + 1 if interleaved else i0 + half
    y = (x[..., i0] + 1j * x[..., i1]) * z[:, None, :]
    x[..., i0], x[..., i1] = y.real, y.imag
    return x


def evict(w, T, keep, first, recent):
    """Kept positions of one (sequence, kv head), ascending."""
    if T <= keep:
        return np.arange(T)
    lo, hi = first, T - recent
    mid = np.arange(lo, hi)
    x = np.where(np.isnan(w[lo:hi]), np.inf, w[lo:hi].astype(np.float64))
    nan = np.isnan(w[lo:hi])
    heavy = mid[np.lexsort((mid, -x, ~nan))][:keep - first - recent]
    return np.sort(np.concatenate([np.arange(lo), heavy, np.arange(hi, T)]))


def verify(target, draft, tokens, counts, ua, us):
    """(accepted, list of token lists), all comparisons in float64."""
    taken, said, at = [], [], 0
    V = target.shape[1]
    for b, n in enumerate(counts):
        j = 0
        while j < n:
            x = int(tokens[at + j])
            if not 0 <= x < V:
                break
            q = float(draft[at + j, x]) if draft is not None else 1.0
            if not float(ua[at + j]) * q < float(target[at + b + j, x]):
                break
            j += 1
        w = target[at + b + j].astype(np.float64)
        if j < n:
            x = int(tokens[at + j])
            rest = w.copy()
            if draft is not None:
                rest = np.maximum(w - draft[at + j].astype(np.float64), 0)
            elif 0 <= x < V:
                rest[x] = 0
            if rest.sum() > 0:
                w = rest
        c = np.cumsum(w)
        over = np.nonzero((c > float(us[b]) * c[-1]) & (w > 0))[0]
        taken.append(j)
        said.append([int(t) for t in tokens[at:at + j]] + [int(over[0]) if c[-1] > 0 else -1])
        at += n
    return taken, said
