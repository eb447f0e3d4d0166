"""Text generation with TANGO over a paged cache, and one training step of its aggregation.

    python examples/generate_tango.py            # prompts in chunks, then token by token
    python examples/generate_tango.py --train    # gradients through norm, rotation, aggregation

The model is the shared-block language model of tango_model_forward (token embedding, one block
applied several times, final RMSNorm, tied logits) with random weights.  Every application
keeps its own pools of key and gate pages; sequences share one page table.  The projections
are plain matrix products; the library appends and aggregates:

    tango_cache_append     k -> norm, rotation -> page;  W_g x -> SiLU -> page;  q -> norm, rotation
    tango_paged_aggregate  u = v * (weighted average of the cached gates)

The generated logits are compared with tango_model_forward over the whole sequences.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import cross_token_gated_gb300 as tg  # noqa: E402

H, D_H, M_H, D, VOCAB, APPS, PAGE = 2, 64, 512, 256, 1024, 3, 16


def make_model(seed=0, dtype=torch.bfloat16, device="cuda"):
    g = torch.Generator().manual_seed(seed)

    def w(out, inner):
        return (torch.randn(out, inner, generator=g) / inner ** 0.5).to(dtype).to(device)

    block = dict(gamma=torch.ones(D, dtype=dtype, device=device), Wq=w(H * D_H, D), Wk=w(H * D_H, D), Wg=w(H * M_H, D),
                 Wv=w(H * M_H, D), Wo=w(D, H * M_H))
    return dict(block=block, embedding=(torch.randn(VOCAB, D, generator=g)).to(dtype).to(device),
                gamma=torch.ones(D, dtype=dtype, device=device), freqs=tg.tg_rope_freqs(D_H, device=device))


def rmsnorm(x, gamma, eps=1e-6):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * gamma.float()).to(x.dtype)


class Server:
    """Sequences over shared pools of pages, one pair of pools per block application."""

    def __init__(self, model, n_seqs, max_len):
        self.model, self.n, self.max_len = model, n_seqs, max_len
        per = -(-max_len // PAGE)
        # any assignment of pages to sequences will do; here they are interleaved
        self.table = torch.arange(n_seqs * per, dtype=torch.int32, device="cuda").reshape(per, n_seqs).t().contiguous()
        self.pools = [tg.cache_pools(n_seqs * per, PAGE, H, D_H, M_H) for _ in range(APPS)]
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")

    def feed(self, chunks):
        """Appends each sequence's new tokens (a list of lists, some may be empty) and returns
        the logits of all of them, in order."""
        model, blk = self.model, self.model["block"]
        counts = [len(c) for c in chunks]
        cu = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
        ids = torch.tensor([t for c in chunks for t in c], device="cuda")
        self.lens += torch.tensor(counts, dtype=torch.int32).cuda()
        h = model["embedding"][ids]
        for k_pages, g_pages in self.pools:
            x = rmsnorm(h, blk["gamma"])
            q, k, raw, v = (x @ blk[n].t() for n in ("Wq", "Wk", "Wg", "Wv"))
            qr, u = torch.empty_like(q), torch.empty_like(v)
            tg.tango_cache_append(q, k, raw, qr, k_pages, g_pages, self.table, cu, self.lens, model["freqs"], H=H)
            tg.tango_paged_aggregate(qr, v, u, k_pages, g_pages, self.table, cu, self.lens, H=H, max_new=max(counts),
                                     max_len=self.max_len)
            h = h + u @ blk["Wo"].t()
        return rmsnorm(h, model["gamma"]) @ model["embedding"].t()


def whole_logits(model, ids):
    """tango_model_forward over one whole sequence."""
    logits = torch.empty(1, len(ids), VOCAB, dtype=torch.bfloat16, device="cuda")
    return tg.tango_model_forward(torch.tensor([ids], dtype=torch.int32, device="cuda"), model["embedding"],
                                  model["gamma"], [model["block"]], logits, H=H, n_apps=APPS)[0]


def generate(prompts, new_tokens, chunk=48, seed=0):
    """Prefills ragged prompts chunk by chunk, then decodes greedily; returns the sequences and
    the largest difference of the last logits from the whole-sequence forward, relative to
    their largest value."""
    model = make_model(seed)
    seqs = [list(p) for p in prompts]
    srv = Server(model, len(seqs), max(len(s) for s in seqs) + new_tokens)
    last = [None] * len(seqs)
    for at in range(0, max(len(s) for s in seqs), chunk):
        part = [s[at:at + chunk] for s in seqs]
        logits, row = srv.feed(part), 0
        for i, c in enumerate(part):
            row += len(c)
            if c:
                last[i] = logits[row - 1]
    for _ in range(new_tokens):
        nxt = [int(row.float().argmax()) for row in last]
        for s, t in zip(seqs, nxt):
            s.append(t)
        last = list(srv.feed([[t] for t in nxt]))
    worst = 0.0
    for s, row in zip(seqs, last):
        want = whole_logits(model, s)[-1].float()
        worst = max(worst, ((row.float() - want).abs().max() / want.abs().max()).item())
    return seqs, worst


def train_step(T=200, seed=0):
    """Gradients of sum(dout * u) from raw q, k, g, v: the aggregation's backward, then that of
    the norm and rotation.  Returns (dq, dk, dg, dv, q's and k's gain gradients)."""
    g = torch.Generator().manual_seed(seed)
    bf = torch.bfloat16

    def normal(width):
        return torch.randn(1, T, width, generator=g).to(bf).cuda()

    q, k, gates, v, dout = normal(H * D_H), normal(H * D_H), normal(H * M_H), normal(H * M_H), normal(H * M_H)
    gain = [(1 + 0.1 * torch.randn(D_H, generator=g)).cuda() for _ in range(2)]
    freqs = tg.tg_rope_freqs(D_H)
    how = dict(H=H, norm=tg.TG_NORM_RMS, q_gain=gain[0], k_gain=gain[1])
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    tg.tango_qk_norm_rope(q, k, qr, kr, freqs, **how)
    out, gbar, den = torch.empty_like(v), torch.empty_like(v), torch.empty(1, H, T, device="cuda")
    tg.tango_aggregate_save(qr, kr, gates, v, out, gbar, den, H=H)
    dqr, dkr, dg, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(v)
    tg.tango_aggregate_backward(qr, kr, gates, v, dout, dqr, dkr, dg, dv, H=H, gbar=gbar, den=den)
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dgain = [torch.empty_like(x) for x in gain]
    tg.tango_qk_norm_rope_backward(q, k, dqr, dkr, dq, dk, freqs, dq_gain=dgain[0], dk_gain=dgain[1], **how)
    return dict(q=q, k=k, g=gates, v=v, dout=dout, gain=gain, dq=dq, dk=dk, dg=dg, dv=dv, dgain=dgain)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--train", action="store_true", help="one backward pass instead of generation")
    args = ap.parse_args()
    if args.train:
        r = train_step()
        print("gradient norms:", {n: round(r[n].float().norm().item(), 4) for n in ("dq", "dk", "dg", "dv")})
        return
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, VOCAB, (n,), generator=g).tolist() for n in (150, 7, 61)]
    seqs, worst = generate(prompts, 12)
    for p, s in zip(prompts, seqs):
        print(f"prompt of {len(p):3d} tokens ->", s[len(p):])
    print(f"last logits against the whole-sequence forward: {worst:.2e} of the largest")


if __name__ == "__main__":
    main()
