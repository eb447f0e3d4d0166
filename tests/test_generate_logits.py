"""The generation example's logits, measured by what the aggregation adds to them.

The logits are tied to the embedding, so that a token's own logit outweighs all others and hides
what the blocks do.  Compared here is, row by row in the 2-norm, the error against the
whole-sequence forward on the scale of that forward's difference from the logits without the
aggregation (u = 0).  An application rounds x, q and k, g, v, the weights, u and the sum to bf16,
about 7 roundings of at most 2^-8 that are independent of one another; 3 applications on both
sides: sqrt(2 * 3 * 7) 2^-8 = 2.5 %.  (Emulated on one side: 0.9 % at most.)  A missing rotation,
uniform weights or a lost page change the same quantity by 14 % and more, which a test without a
GPU confirms on the same model and tokens.
"""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

TOL = math.sqrt(2 * 3 * 7) * 2.0 ** -8
PROMPTS, NEW = (150, 7, 61), 6


def _tokens(ex):
    """Three sequences of fixed tokens: prompts and what follows them."""
    g = torch.Generator().manual_seed(5)
    return [torch.randint(0, ex.VOCAB, (n + NEW,), generator=g).tolist() for n in PROMPTS]


def _forward(ex, model, ids, rnd=lambda x: x, rotate=True, tau=10.0, lost=None, update=True):
    """The example's model over one sequence in float64, intermediates through rnd."""
    H, DH, T = ex.H, ex.D_H, len(ids)
    w = {k: t.double() for k, t in model["block"].items()}
    E = model["embedding"].double()
    ang = torch.arange(T, dtype=torch.float64)[:, None, None] * 10000.0 ** (-torch.arange(0, DH, 2, dtype=torch.float64) / DH)
    c, s = ang.cos(), ang.sin()

    def rms(x):
        return rnd(x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt())

    def unit(x):
        x = x.view(T, H, DH)
        x = x / x.norm(dim=-1, keepdim=True)
        a, b = x[..., :DH // 2], x[..., DH // 2:]
        return rnd(torch.cat([a * c - b * s, a * s + b * c], -1) if rotate else x)

    h = E[ids]
    for _ in range(ex.APPS if update else 0):
        x = rms(h)
        q, k = unit(rnd(x @ w["Wq"].T)), unit(rnd(x @ w["Wk"].T))
        g = rnd(x @ w["Wg"].T)
        g, v = rnd(g * torch.sigmoid(g)).view(T, H, -1), rnd(x @ w["Wv"].T).view(T, H, -1)
        p = rnd(torch.exp(tau * (torch.einsum("ihd,jhd->hij", q, k) - 1))).tril()
        if lost is not None:
            p[:, lost.stop:, lost] = 0
        u = rnd(torch.einsum("hij,jhc->ihc", p / p.sum(-1, keepdim=True), g) * v).flatten(1)
        h = rnd(h + u @ w["Wo"].T)
    return rnd(rms(h) @ E.T)


def _errors(got, want, base):
    """Per row: the 2-norm of the error over that of what the blocks add."""
    return (got - want).norm(dim=1) / (want - base).norm(dim=1)


def test_the_measure_sees_what_it_has_to(lib):
    """bf16 roundings stay inside the tolerance, mistakes of the aggregation far outside."""
    import generate_tango as ex
    model = ex.make_model(device="cpu")
    for ids in _tokens(ex):
        want, base = _forward(ex, model, ids), _forward(ex, model, ids, update=False)
        assert _errors(_forward(ex, model, ids, rnd=lambda x: x.bfloat16().double()), want, base).max() <= TOL / math.sqrt(2)
        for wrong in (dict(rotate=False), dict(tau=0.0), dict(lost=slice(0, min(len(ids) // 2, ex.PAGE)))):
            err = _errors(_forward(ex, model, ids, **wrong), want, base)
            assert err[-1] > 4 * TOL and (err > 4 * TOL).sum() >= len(ids) // 2 - 1, wrong


@pytest.mark.gpu
@pytest.mark.parametrize("cuts", [[48, 48, 48, 6], [1, 7, 60, 82], [150]], ids=["chunks", "uneven", "whole"])
def test_every_new_token_follows_the_whole_sequence_forward(cuts):
    """Prompts in chunks, then token by token with given tokens: all rows' logits."""
    import generate_tango as ex
    model, seqs = ex.make_model(), _tokens(ex)
    srv = ex.Server(model, len(seqs), max(len(s) for s in seqs))
    got, at = [[] for _ in seqs], 0
    for n in cuts:
        parts = [s[:p][at:at + n] for s, p in zip(seqs, PROMPTS)]
        rows = srv.feed(parts).split([len(p) for p in parts])
        got, at = [a + [r] for a, r in zip(got, rows)], at + n
    for i in range(NEW):
        rows = srv.feed([[s[p + i]] for s, p in zip(seqs, PROMPTS)])
        got = [a + [r[None]] for a, r in zip(got, rows)]
    for ids, rows in zip(seqs, got):
        want = ex.whole_logits(model, ids).double()
        base = (ex.rmsnorm(model["embedding"][ids], model["gamma"]) @ model["embedding"].t()).double()
        err = _errors(torch.cat(rows).double(), want, base)
        assert err.shape[0] == len(ids) and err.max().item() <= TOL, err.max().item()
