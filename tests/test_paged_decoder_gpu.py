"""The whole decoder from the library's own operations on a paged cache: streams of their own lengths go through it in ragged
chunks, then in drafted and single tokens, and their logits are those of the oracle and of Model with a cache for each."""
import numpy as np
import pytest
import torch

import synth
from oracle import ms_oracle as O

pytestmark = pytest.mark.gpu
ms = pytest.importorskip("decoder_only_transformer_int4_b200")

PAGE, CAPACITY = 16, 160
TOL = 2e-3     # as for the model's own paths


class PagedDecoder:
    """Layers of matmul_w4, rope_append_paged, attn_paged, skip_layernorm and the LM head over one table for all layers."""

    def __init__(self, draw, batch, kv_type, seed):
        sh, dev = draw.shape, "cuda"
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).float().to(dev)  # noqa: E731
        self.sh, self.batch = sh, batch
        self.layers = [([up(x) for x in (l.ln1_g, l.ln1_b, l.ln2_g, l.ln2_b)], [ms.quantize_int4_g32(up(w)) for w in l.w])
                       for l in draw.layers]
        self.emb, self.head, self.fg, self.fb = up(draw.tok_emb), up(draw.lm_head), up(draw.ln_f_g), up(draw.ln_f_b)
        self.freq = torch.tensor([sh.rope_base ** (-2 * j / sh.head_dim) for j in range(sh.head_dim // 2)], dtype=torch.float64, device=dev)
        pages = batch * CAPACITY // PAGE
        g = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(pages, generator=g).to(torch.int32).reshape(batch, -1).cuda()
        self.lens = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        shape = (pages, sh.n_kv_heads, PAGE, sh.head_dim)
        self.kv = [ms.PagedKV(torch.full(shape, float("nan"), dtype=kv_type, device=dev), torch.full(shape, float("nan"), dtype=kv_type, device=dev),
                              self.table, self.lens, self.status) for _ in self.layers]

    def run(self, tokens):
        """tokens: a list of new tokens for each stream; logits of all rows, packed."""
        sh, counts = self.sh, [len(t) for t in tokens]
        H, hk, hd = sh.n_heads, sh.n_kv_heads, sh.head_dim
        start = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
        self.lens += torch.tensor(counts, dtype=torch.int32).cuda()
        x, y = self.emb[torch.tensor(sum(tokens, []), device="cuda")].clone(), None
        n = x.shape[0]
        for kv, ((g1, b1, g2, b2), w) in zip(self.kv, self.layers):
            qkv = ms.matmul_w4(ms.skip_layernorm(x, y, g1, b1, sh.ln_eps), *w[0]).view(n, H + 2 * hk, hd)
            q = ms.rope_append_paged(kv, qkv[:, :H], qkv[:, H:H + hk], qkv[:, H + hk:], start, self.freq)
            a = ms.attn_paged(kv, q, start, max(counts))
            h = ms.skip_layernorm(x, ms.matmul_w4(a.view(n, H * hd), *w[1]), g2, b2, sh.ln_eps)
            y = ms.matmul_w4(torch.nn.functional.gelu(ms.matmul_w4(h, *w[2])), *w[3])
        parts = [ms.lm_head_argmax(r, self.head, self.fg, self.fb, sh.ln_eps) for r in (x + y).split(64)]
        ms.op_status(self.status)
        return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])

    def drop(self, counts):
        """Takes back the last positions of each stream (refused drafts)."""
        self.lens -= torch.tensor(counts, dtype=torch.int32).cuda()


@pytest.mark.parametrize("kv_type,store", [(torch.float32, "fp32"), (torch.float16, "fp16")])
@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (8, 2)])
def test_a_decoder_of_the_paged_operators(kv_type, store, heads, kv_heads):
    sh = synth.Shape("paged", 2, heads * 64, heads, kv_heads, 512, vocab=1393)
    draw = synth.make_weights(sh, seed=5, std=0.05, ln_random=True)
    om = O.OracleModel(draw, "int4", kv_store=store)
    model = ms.Model.from_draw(draw, "int4")
    rng = np.random.default_rng(7)
    prompts = [list(map(int, rng.integers(0, sh.vocab, n))) for n in (97, 1, 40)]
    dec = PagedDecoder(draw, len(prompts), kv_type, seed=6)
    # the prompts in ragged chunks of at most 64 rows
    cuts = [[(0, 30), (30, 94), (94, 97)], [(0, 0), (0, 0), (0, 1)], [(0, 17), (17, 18), (18, 40)]]
    logits = [np.zeros((0, sh.vocab))] * 3
    for step in range(3):
        out, best = dec.run([p[slice(*c[step])] for p, c in zip(prompts, cuts)])
        rows = np.split(out.cpu().numpy(), np.cumsum([c[step][1] - c[step][0] for c in cuts])[:-1])
        logits = [np.concatenate([a, b]) for a, b in zip(logits, rows)]
    want = [om.teacher_forced(None, p) for p in prompts]
    for got, ref in zip(logits, want):
        assert np.abs(got - ref).max() <= TOL
    # greedy steps with drafts: what the target takes is what Model decodes one by one
    text = [p + [int(ref[-1].argmax())] for p, ref in zip(prompts, want)]
    model_text = []
    for p in prompts:
        cache = ms.Cache(model, 1, CAPACITY, **({"kv_format": ms.MS_KV_F16} if store == "fp16" else {}))
        _, am = cache.prefill(torch.tensor([p], dtype=torch.int64, device="cuda"), None)
        toks, _ = cache.generate(12)
        model_text.append(p + [int(am.item())] + [int(t) for t in toks.cpu().numpy()[:, 0]])
    one = torch.nn.functional.one_hot
    for step in range(4):
        # the right next tokens as drafts, one of them spoilt
        drafts = [m[len(t):len(t) + n] for t, m, n in zip(text, model_text, (3, 0, 2))]
        if drafts[0]:
            spoilt = step % len(drafts[0])
            drafts[0][spoilt] = (drafts[0][spoilt] + 1) % sh.vocab
        out, best = dec.run([[t[-1]] + d for t, d in zip(text, drafts)])
        n = [len(d) for d in drafts]
        dstart = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32).cuda()
        flat = torch.tensor(sum(drafts, []), dtype=torch.int32).cuda()
        taken, tokens = ms.verify_draft(one(best.long(), sh.vocab).float(), None, flat, dstart, 3,
                                        torch.full((sum(n),), 0.5, device="cuda"), torch.full((3,), 0.5, device="cuda"), dec.status)
        ms.op_status(dec.status)
        dec.drop([k - int(a) for k, a in zip(n, taken.tolist())])
        for i, row in enumerate(tokens.tolist()):
            said = [t for t in row if t >= 0]
            assert len(said) == taken[i].item() + 1
            text[i] += said
    assert all(len(t) >= len(p) + 5 for t, p in zip(text, prompts))
    for t, m, p in zip(text, model_text, prompts):
        ref = om.teacher_forced(None, t[:-1])
        for j in range(len(p), min(len(t), len(m))):
            # the same tokens as long as no two logits are closer than the tolerance
            if t[j] != m[j]:
                assert O.top2_margin(ref[j - 1:j]).item() <= 2 * TOL
                break
