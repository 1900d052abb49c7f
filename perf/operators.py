"""Measured cases of the paged-cache operators: rotary positions with the append into the pages, attention of
the newest tokens over the pages, eviction by accumulated attention weight, and verification of drafted tokens.

`run` makes one pass through an operator: with `own` false in its plain form (elementary torch operations in
32 bits, 64 where positions, long sums or borders need them), with `own` true by the library's entry point.

Shared layout: K and V pages [n_pages, kv_heads, page, head_dim]; `table` int32 [batch, max_pages] gives the
page that holds positions page*j .. page*j + page - 1 of a sequence; `lens` int32 [batch] counts the positions
held, the newest rows included; the rows of a call are packed, those of sequence b at row_start[b] ..
row_start[b+1] - 1, and are the last positions of their sequence.
"""
import json
import math
import random

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---- cases --------------------------------------------------------------------------------

def listed():
    return [
        # 64 streams of the medium decoder each append one token to the half-precision cache
        dict(name="rope, 64 streams, one token", op="rope", batch=64, heads=16, kv_heads=4, head_dim=64, rot=64,
             interleaved=False, scaling="none", q="f32", kv="f16", page=16, base_lo=504, base_hi=1016, rows_lo=1, rows_hi=1),
        # eight prompts of odd lengths, interleaved pairs on half of each head, positions squeezed by four
        dict(name="rope, eight ragged prompts", op="rope", batch=8, heads=32, kv_heads=8, head_dim=128, rot=64,
             interleaved=True, scaling="linear", q="bf16", kv="bf16", page=64, base_lo=0, base_hi=257, rows_lo=301, rows_hi=701),
        # a long prompt's second half, far positions, frequencies blended for a context 16 times the trained one
        dict(name="rope, long prompt, far positions", op="rope", batch=1, heads=24, kv_heads=8, head_dim=64, rot=64,
             interleaved=False, scaling="blend", q="f32", kv="f16", page=128, base_lo=65529, base_hi=65529, rows_lo=32767, rows_hi=32767),
        # one stream of the medium decoder at the end of its prompt, fp32 cache: the smallest call
        dict(name="attn, one stream, fp32", op="attn", batch=1, heads=16, kv_heads=4, head_dim=64, q="f32", kv="f32",
             page=16, len_lo=577, len_hi=577, rows_lo=1, rows_hi=1, weights=False),
        # 64 streams of the medium decoder, half cache, fp32 activations, weights accumulated for the eviction
        dict(name="attn, 64 streams, weights", op="attn", batch=64, heads=16, kv_heads=4, head_dim=64, q="f32", kv="f16",
             page=16, len_lo=505, len_hi=1024, rows_lo=1, rows_hi=1, weights=True),
        # 16 sequences of very different lengths, one to six newest tokens each (drafts to verify)
        dict(name="attn, drafted rows, ragged", op="attn", batch=16, heads=32, kv_heads=8, head_dim=128, q="bf16", kv="bf16",
             page=64, len_lo=1021, len_hi=16411, rows_lo=1, rows_hi=6, weights=False),
        # one sequence with a very long cache: the work has to be split over its length
        dict(name="attn, one long cache", op="attn", batch=1, heads=24, kv_heads=8, head_dim=64, q="f16", kv="f16",
             page=128, len_lo=131071, len_hi=131071, rows_lo=1, rows_hi=1, weights=False),
        # 64 streams of the medium decoder cut back to 512 positions
        dict(name="evict, 64 streams", op="evict", batch=64, kv_heads=4, head_dim=64, kv="f16", page=16, len_lo=505,
             len_hi=1024, keep=512, first=4, recent=128),
        # four long sequences cut back to an eighth or so of their length
        dict(name="evict, long caches", op="evict", batch=4, kv_heads=8, head_dim=128, kv="bf16", page=64, len_lo=8190,
             len_hi=32771, keep=4099, first=0, recent=1024),
        # one stream verifies four drafted tokens over the decoder's vocabulary
        dict(name="verify, one stream", op="verify", batch=1, vocab=1393, drafts_lo=4, drafts_hi=4, draft_probs=True),
        # 64 streams, nought to eight drafts each
        dict(name="verify, 64 streams", op="verify", batch=64, vocab=32003, drafts_lo=0, drafts_hi=8, draft_probs=True),
        # a large vocabulary, drafts taken without probabilities (looked up in the text so far)
        dict(name="verify, large vocabulary", op="verify", batch=32, vocab=100003, drafts_lo=1, drafts_hi=5, draft_probs=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 5, 8])
    return kv * rng.choice([1, 2, 3, 4, 6, 7, 8]), kv


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "evict", "verify"])
    heads, kv_heads = _heads(rng)
    head_dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    q, kv = rng.choice([("f32", "f32"), ("f32", "f16"), ("f16", "f16"), ("bf16", "bf16")])
    if op == "rope":
        batch = _log(rng, 1, 64)
        rows = _log(rng, 1, max(1, 24000000 // (batch * (heads + 2 * kv_heads) * head_dim)))
        rows = min(rows, 32000)
        base = _log(rng, 1, 65536)
        rot = rng.choice([head_dim, head_dim, head_dim // 2, 2 * rng.randrange(1, head_dim // 2 + 1)])
        return dict(op=op, batch=batch, heads=heads, kv_heads=kv_heads, head_dim=head_dim, rot=rot,
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "blend"]), q=q, kv=kv,
                    page=page, base_lo=base // 3, base_hi=base, rows_lo=(rows + 1) // 2, rows_hi=rows)
    if op == "attn":
        batch = _log(rng, 1, 96)
        most = 240000000 // (batch * kv_heads * head_dim * BYTES[kv])
        length = _log(rng, 17, max(20, min(most, 131072)))
        rows = rng.choice([1, 1, 1, 2, 4, 7])
        return dict(op=op, batch=batch, heads=heads, kv_heads=kv_heads, head_dim=head_dim, q=q, kv=kv, page=page,
                    len_lo=rng.choice([0, 1 + length // 8, length]), len_hi=length, rows_lo=1, rows_hi=rows,
                    weights=rng.random() < 0.4)
    if op == "evict":
        batch = _log(rng, 1, 64)
        most = 160000000 // (batch * kv_heads * head_dim * BYTES[kv])
        length = _log(rng, 64, max(80, min(most, 32768)))
        keep = max(8, int(length * rng.uniform(0.1, 0.9)))
        return dict(op=op, batch=batch, kv_heads=kv_heads, head_dim=head_dim, kv=kv, page=page, len_lo=length // 3,
                    len_hi=length, keep=keep, first=rng.choice([0, 1, 4]), recent=rng.randrange(0, keep - 4))
    vocab = _log(rng, 300, 130000)
    batch = _log(rng, 1, max(1, min(96, 3600000 // vocab)))
    drafts = rng.randrange(1, 9)
    return dict(op="verify", batch=batch, vocab=vocab, drafts_lo=rng.randrange(0, drafts + 1), drafts_hi=drafts,
                draft_probs=rng.random() < 0.7)


def _sizes(case):
    """Lengths and newest rows of each sequence: a property of the case, whatever the seed."""
    r = random.Random(json.dumps({k: v for k, v in case.items() if k != "name"}, sort_keys=True))
    n = case["batch"]
    if case["op"] == "verify":
        return None, [r.randint(case["drafts_lo"], case["drafts_hi"]) for _ in range(n)]
    if case["op"] == "rope":
        rows = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(n)]
        return [r.randint(case["base_lo"], case["base_hi"]) + x for x in rows], rows
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(n)]
    return lens, [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(n)] if case["op"] == "attn" else None


def work(case):
    """Bytes that have to be read and written, and multiply-adds twice over."""
    lens, rows = _sizes(case)
    if case["op"] == "verify":
        # the acceptance reads one value of each matrix for a draft; the choice reads one row of each
        return {"bytes": case["batch"] * case["vocab"] * 4 * (2 if case["draft_probs"] else 1) + 32 * sum(rows), "flops": 0}
    hk, hd, kb = case["kv_heads"], case["head_dim"], BYTES[case["kv"]]
    if case["op"] == "rope":
        n, qb = sum(rows), BYTES[case["q"]]
        return {"bytes": n * hd * (2 * case["heads"] * qb + 2 * hk * (qb + kb)), "flops": 3 * n * (case["heads"] + hk) * case["rot"]}
    if case["op"] == "attn":
        b = sum(lens) * hk * hd * 2 * kb + 2 * sum(rows) * case["heads"] * hd * BYTES[case["q"]]
        return {"bytes": b + (8 * hk * sum(lens) if case["weights"] else 0),
                "flops": 4 * case["heads"] * hd * sum(n * t for n, t in zip(rows, lens))}
    kept = sum(min(t, case["keep"]) for t in lens)
    return {"bytes": 4 * hk * sum(lens) + 4 * kept * hk * hd * kb + 8 * hk * kept, "flops": 0}


# ---- inputs -------------------------------------------------------------------------------

def _inv_freq(rot, scaling):
    """Angle per position of each pair, in double.  linear: positions squeezed by 4.  blend: pairs that turn
    fewer than once within 4096 positions are slowed 16 times, those that turn more than 32 times are left,
    those between are mixed in proportion."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        return f / 4, 1.0
    if scaling == "blend":
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        return f * keep + f / 16 * (1 - keep), 0.1 * math.log(16.0) + 1
    return f, 1.0


def _pages(counts, page, gen, dev):
    """Tables for sequences of the given lengths (several lists of them share one pool) and the pool's size."""
    need = [[-(-t // page) for t in c] for c in counts]
    total = sum(map(sum, need)) + 3
    ids, at, tables = torch.randperm(total, generator=gen, device=dev).to(torch.int32), 0, []
    for n in need:
        t = torch.zeros((len(n), max(1, max(n))), dtype=torch.int32, device=dev)
        for b, k in enumerate(n):
            t[b, :k] = ids[at:at + k]
            at += k
        tables.append(t)
    return tables, total


def _starts(rows, dev):
    return torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(shape, kind, scale=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * scale).to(TYPES[kind])

    lens, rows = _sizes(case)
    s = dict(case)
    if case["op"] == "verify":
        n, v, batch = sum(rows), case["vocab"], case["batch"]
        s["row_start"] = _starts(rows, dev)
        s["most"] = max(rows)
        logits = torch.randn((n + batch, v), generator=gen, device=dev) * 3
        s["target"] = torch.softmax(logits, 1)
        own_row = torch.tensor([r + b for b, (a, c) in enumerate(zip(np.cumsum([0] + rows), rows)) for r in range(a, a + c)],
                               dtype=torch.int64, device=dev)
        near = logits[own_row] + torch.randn((n, v), generator=gen, device=dev) * 0.7   # the draft model's view
        probs = torch.softmax(near, 1)
        s["tokens"] = torch.multinomial(probs, 1, generator=gen)[:, 0].to(torch.int32) if n else \
            torch.zeros((0,), dtype=torch.int32, device=dev)
        if not case["draft_probs"] and n:
            s["tokens"] = probs.argmax(1).to(torch.int32)
        s["draft"] = probs.contiguous() if case["draft_probs"] else None
        s["u_accept"] = torch.rand((n,), generator=gen, device=dev)
        s["u_sample"] = torch.rand((batch,), generator=gen, device=dev)
        return s
    page, hk, hd = case["page"], case["kv_heads"], case["head_dim"]
    kept = [[min(t, case["keep"]) for t in lens]] if case["op"] == "evict" else []
    tables, pool = _pages([lens] + kept, page, gen, dev)
    s["table"] = tables[0]
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["k"] = normal((pool, hk, page, hd), case["kv"])
    s["v"] = normal((pool, hk, page, hd), case["kv"])
    cap = tables[0].shape[1] * page
    if case["op"] == "evict":
        s["dst"] = tables[1]
        w = torch.exp(2 * torch.randn((case["batch"], hk, cap), generator=gen, device=dev) - 4)
        # some positions were never looked at: their weight is 0, and they tie
        s["weights"] = torch.where(torch.rand(w.shape, generator=gen, device=dev) < 0.1, torch.zeros_like(w), w)
        s["weights"] *= (torch.arange(cap, device=dev) < s["lens"][:, None, None])
        return s
    n, heads = sum(rows), case["heads"]
    s["row_start"] = _starts(rows, dev)
    if case["op"] == "rope":
        s["inv_freq"], s["mscale"] = _inv_freq(case["rot"], case["scaling"])
        s["inv_freq"] = s["inv_freq"].to(dev)
        qkv = normal((n, heads + 2 * hk, hd), case["q"])   # one fused row per token, as the projection leaves it
        s["q_in"], s["k_in"], s["v_in"] = qkv[:, :heads], qkv[:, heads:heads + hk], qkv[:, heads + hk:]
        return s
    s["most"] = max(rows)
    s["q_in"] = normal((n, heads, hd), case["q"], 2.0)
    s["scale"] = hd ** -0.5
    s["weights"] = torch.rand((case["batch"], hk, cap), generator=gen, device=dev) if case["weights"] else None
    return s


# ---- one pass -----------------------------------------------------------------------------

def _owner(s, n):
    """Sequence and place within it of each of the n packed rows."""
    t = torch.arange(n, device=s["row_start"].device, dtype=torch.int32)
    b = torch.searchsorted(s["row_start"][1:].contiguous(), t, right=True)
    return b, t - s["row_start"][b]


def _plain_rope(s):
    q, k, v = s["q_in"], s["k_in"], s["v_in"]
    b, i = _owner(s, q.shape[0])
    pos = (s["lens"][b] - (s["row_start"][b + 1] - s["row_start"][b]) + i).long()
    ang = pos.double()[:, None, None] * s["inv_freq"]
    cos, sin = (torch.cos(ang) * s["mscale"]).float(), (torch.sin(ang) * s["mscale"]).float()
    rot = s["rot"]

    def turn(x):
        x = x.float()
        r = x[..., :rot]
        if s["interleaved"]:
            a, c = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - c * sin, a * sin + c * cos), -1).flatten(-2)
        else:
            a, c = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat((a * cos - c * sin, a * sin + c * cos), -1)
        return torch.cat((r, x[..., rot:]), -1)

    pages, at = s["table"][b, pos // s["page"]].long(), pos % s["page"]
    s["k"][pages, :, at] = turn(k).to(s["k"].dtype)
    s["v"][pages, :, at] = v.float().to(s["v"].dtype)
    return {"q": turn(q).to(q.dtype), "k": s["k"], "v": s["v"]}


def _plain_attn(s):
    q, table, lens, most = s["q_in"], s["table"], s["lens"], s["most"]
    n, heads, hd = q.shape
    batch, hk, page = table.shape[0], s["kv_heads"], s["page"]
    cap = table.shape[1] * page
    kk = s["k"][table.long()].permute(0, 2, 1, 3, 4).reshape(batch, hk, cap, hd).float()
    vv = s["v"][table.long()].permute(0, 2, 1, 3, 4).reshape(batch, hk, cap, hd).float()
    b, i = _owner(s, n)
    padded = torch.zeros((batch, most, heads, hd), device=q.device)
    padded[b, i.long()] = q.float()
    g = heads // hk
    qq = padded.reshape(batch, most, hk, g, hd).permute(0, 2, 1, 3, 4).reshape(batch, hk, most * g, hd)
    sc = (qq @ kk.transpose(2, 3)) * s["scale"]
    count = s["row_start"][1:] - s["row_start"][:-1]
    place = torch.arange(most, device=q.device, dtype=torch.int32)
    last = (lens - count)[:, None] + place                        # position of each row
    seen = (torch.arange(cap, device=q.device) <= last[..., None]) & (place < count[:, None])[..., None]
    seen = seen[:, None, :, None].expand(batch, hk, most, g, cap).reshape(batch, hk, most * g, cap)
    sc = sc.masked_fill(~seen, float("-inf"))
    top = sc.amax(3, keepdim=True)
    p = torch.exp(sc - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    p = p / p.sum(3, keepdim=True).clamp_min(torch.finfo(torch.float32).tiny)
    o = (p @ vv).reshape(batch, hk, most, g, hd).permute(0, 2, 1, 3, 4).reshape(batch, most, heads, hd)
    out = {"out": o[b, i.long()].to(q.dtype)}
    if s["weights"] is not None:
        s["weights"] += p.sum(2)
        out["weights"] = s["weights"]
    return out


def _plain_evict(s):
    w, lens, page, keep = s["weights"], s["lens"], s["page"], s["keep"]
    batch, hk, cap = w.shape
    pos = torch.arange(cap, device=w.device)
    t = lens[:, None, None]
    guarded = (pos < s["first"]) | (pos >= t - s["recent"]) | (t <= keep)
    key = torch.where(guarded, torch.full_like(w, float("inf")), w)
    key = torch.where(pos < t, key, torch.full_like(w, float("-inf")))
    order = torch.sort(key, dim=2, descending=True, stable=True).indices[:, :, :keep]
    order = torch.cat((order, order.new_full((batch, hk, keep - order.shape[2]), cap)), 2)
    kept = torch.sort(torch.where(order < t, order, torch.full_like(order, cap)), dim=2).values
    real = kept < t
    src = torch.where(real, kept, torch.zeros_like(kept))
    bi = torch.arange(batch, device=w.device)[:, None, None]
    gi = torch.arange(hk, device=w.device)[None, :, None]
    j = torch.arange(keep, device=w.device)[None, None, :].expand_as(kept)
    j = torch.where(real, j, torch.zeros_like(j))
    from_page, to_page = s["table"].long()[bi, src // page], s["dst"].long()[bi, j // page]
    head = kept[:, :, :1].clamp_max(cap - 1)
    head_page = s["table"].long()[bi, head // page]

    def move(x):   # a place without a row of its own repeats the first one
        rows = torch.where(real[..., None], x[from_page, gi, src % page], x[head_page, gi, head % page])
        x[to_page, gi, j % page] = rows

    move(s["k"])
    move(s["v"])
    new = torch.zeros_like(w)
    some = min(keep, cap)
    taken = torch.gather(w, 2, kept[:, :, :some].clamp_max(cap - 1))
    new[:, :, :some] = torch.where(real[:, :, :some], taken, torch.zeros_like(taken))
    kept = torch.where(real, kept, torch.full_like(kept, -1)).to(torch.int32)
    return {"k": s["k"], "v": s["v"], "weights": new, "kept": kept, "lens": torch.minimum(lens, torch.full_like(lens, keep))}


def _plain_verify(s):
    target, draft, tok, start, most = s["target"], s["draft"], s["tokens"], s["row_start"], s["most"]
    batch, v = s["batch"], s["vocab"]
    count = (start[1:] - start[:-1]).long()
    place = torch.arange(most, device=target.device)
    real = place < count[:, None]
    row = start[:-1, None].long() + torch.where(real, place, torch.zeros_like(place))
    bi = torch.arange(batch, device=target.device)
    if tok.shape[0]:
        row = row.clamp_max(tok.shape[0] - 1)
        x = tok[row].long()
        p = target[(row + bi[:, None]), x].double()
        q = draft[row, x].double() if draft is not None else torch.ones_like(p)
        yes = (s["u_accept"][row].double() * q < p) & real
        taken = torch.cumprod(yes.long(), 1).sum(1)
    else:
        x, taken = torch.zeros((batch, most), dtype=torch.long, device=target.device), torch.zeros_like(count)
    at = start[:-1].long() + taken
    w = target[at + bi].double()
    refused = (taken < count)[:, None]
    if tok.shape[0]:
        at = at.clamp_max(tok.shape[0] - 1)
        if draft is not None:
            less = draft[at].double()
        else:
            less = torch.zeros_like(w).scatter_(1, tok[at].long()[:, None], float("inf"))
        rest = (w - less).clamp_min(0)
        rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, w)
        w = torch.where(refused, rest, w)
    cdf = torch.cumsum(w, 1)
    nxt = (cdf <= s["u_sample"].double()[:, None] * cdf[:, -1:]).sum(1)
    wide = torch.arange(most + 1, device=target.device)
    said = torch.cat((x, x.new_zeros((batch, 1))), 1)
    said = torch.where(wide < taken[:, None], said, torch.where(wide == taken[:, None], nxt[:, None], torch.full_like(said, -1)))
    return {"accepted": taken.to(torch.int32), "tokens": said.to(torch.int32)}


def _own(s):
    import decoder_only_transformer_int4_b200 as ms
    if s["op"] == "verify":
        taken, said = ms.verify_draft(s["target"], s["draft"], s["tokens"], s["row_start"], s["most"], s["u_accept"], s["u_sample"])
        return {"accepted": taken, "tokens": said}
    kv = ms.PagedKV(s["k"], s["v"], s["table"], s["lens"])
    if s["op"] == "rope":
        q = ms.rope_append_paged(kv, s["q_in"], s["k_in"], s["v_in"], s["row_start"], s["inv_freq"],
                                 interleaved=s["interleaved"], mscale=s["mscale"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    if s["op"] == "attn":
        out = {"out": ms.attn_paged(kv, s["q_in"], s["row_start"], s["most"], scale=s["scale"], weights=s["weights"])}
        return out if s["weights"] is None else {**out, "weights": s["weights"]}
    kept, new, lens = ms.evict_paged(kv, s["weights"], s["dst"], s["keep"], first=s["first"], recent=s["recent"])
    return {"k": s["k"], "v": s["v"], "weights": new, "kept": kept, "lens": lens}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "rope":
        return _plain_rope(state)
    if state["op"] == "attn":
        return _plain_attn(state)
    return _plain_evict(state) if state["op"] == "evict" else _plain_verify(state)


# ---- the definitions in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    lens, rows = _sizes(case)
    if case["op"] == "verify":
        return _exact_verify(s, rows)
    if case["op"] == "evict":
        return _exact_evict(s, lens)
    hk, page = case["kv_heads"], case["page"]
    starts = np.concatenate([[0], np.cumsum(rows)])
    k, v = s["k"].double(), s["v"].double()
    table = s["table"].long()
    if case["op"] == "attn":
        out = torch.empty(s["q_in"].shape, dtype=torch.float64, device=k.device)
        weights = None if s["weights"] is None else s["weights"].double()
        g = case["heads"] // hk
        for b, (t, n) in enumerate(zip(lens, rows)):
            pages = table[b, :-(-t // page)]
            for h in range(hk):
                kb, vb = (x[pages, h].reshape(-1, case["head_dim"])[:t] for x in (k, v))
                for i in range(n):
                    upto = max(0, t - n + i + 1)
                    qb = s["q_in"][starts[b] + i, h * g:(h + 1) * g].double()
                    p = torch.softmax((qb * s["scale"]) @ kb[:upto].T, 1)
                    out[starts[b] + i, h * g:(h + 1) * g] = p @ vb[:upto]
                    if weights is not None:
                        weights[b, h, :upto] += p.sum(0)
        return {"out": out, "weights": weights} if weights is not None else {"out": out}
    half, rot = case["rot"] // 2, case["rot"]
    first = torch.arange(half, device=k.device) * 2 if case["interleaved"] else torch.arange(half, device=k.device)
    second = first + (1 if case["interleaved"] else half)
    q = s["q_in"].double().clone()
    for b, (t, n) in enumerate(zip(lens, rows)):
        pos = torch.arange(t - n, t, device=k.device)
        z = torch.polar(torch.full((n, 1, half), float(s["mscale"]), dtype=torch.float64, device=k.device),
                        pos.double()[:, None, None] * s["inv_freq"])
        here = slice(int(starts[b]), int(starts[b + 1]))
        for src, put in ((s["q_in"], "q"), (s["k_in"], "k")):
            x = src[here].double()
            y = torch.complex(x[..., first], x[..., second]) * z
            x = x.clone()
            x[..., first], x[..., second] = y.real, y.imag
            if put == "q":
                q[here] = x
            else:
                k[table[b, pos // page], :, pos % page] = x
        v[table[b, pos // page], :, pos % page] = s["v_in"][here].double()
    return {"q": q, "k": k, "v": v}


def _exact_evict(s, lens):
    page, keep, hk = s["page"], s["keep"], s["kv_heads"]
    k, v = s["k"].double(), s["v"].double()
    w = s["weights"].cpu().numpy().astype(np.float64)
    new, kept = np.zeros_like(w), np.full((len(lens), hk, keep), -1, np.int32)
    table, dst = s["table"].long(), s["dst"].long()
    for b, t in enumerate(lens):
        for h in range(hk):
            if t <= keep:
                ids = np.arange(t)
            else:
                lo, hi = min(s["first"], t), max(t - s["recent"], min(s["first"], t))
                middle = np.arange(lo, hi)
                heavy = middle[np.lexsort((middle, -w[b, h, lo:hi]))][:keep - (t - len(middle))]
                ids = np.sort(np.concatenate([np.arange(lo), heavy, np.arange(hi, t)]))
            m = len(ids)
            kept[b, h, :m] = ids
            new[b, h, :m] = w[b, h, ids]
            at, to = torch.from_numpy(ids).to(k.device), torch.arange(m, device=k.device)
            for x in (k, v):
                x[dst[b, to // page], h, to % page] = x[table[b, at // page], h, at % page]
    return {"k": k, "v": v, "weights": new, "kept": kept, "lens": np.minimum(np.array(lens), keep).astype(np.int32)}


def _exact_verify(s, rows):
    target = s["target"].cpu().numpy()
    draft = None if s["draft"] is None else s["draft"].cpu().numpy()
    tok, ua, us = (s[n].cpu().numpy() for n in ("tokens", "u_accept", "u_sample"))
    taken = np.zeros(len(rows), np.int32)
    said = np.full((len(rows), s["most"] + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(rows):
        j = 0
        while j < n:
            x = tok[at + j]
            chance = float(target[at + b + j, x]) / (float(draft[at + j, x]) if draft is not None else 1.0)
            if not float(ua[at + j]) < chance:
                break
            said[b, j] = x
            j += 1
        w = target[at + b + j].astype(np.float64)
        if j < n:
            rest = w.copy()
            if draft is not None:
                rest = np.maximum(w - draft[at + j], 0.0)
            else:
                rest[tok[at + j]] = 0.0
            if rest.sum() > 0:
                w = rest
        c = np.cumsum(w)
        taken[b] = j
        said[b, j] = int(np.searchsorted(c, float(us[b]) * c[-1], side="right"))
        at += n
    return {"accepted": taken, "tokens": said}
