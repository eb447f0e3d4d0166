"""The generation example: append and aggregation as a serving loop uses them, and the
gradients of norm, rotation and aggregation together."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_generation_follows_the_whole_sequence_forward():
    """Chunked prompts and single tokens over the cache give the whole-sequence logits.  Both
    round x, q, k, g, v, u and the residual to bf16 (2^-8 each) in three applications, about 7
    roundings of the update in each; their sum stays well under 7 * 3 * 2^-8 of the scale."""
    import generate_tango as ex
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, ex.VOCAB, (n,), generator=g).tolist() for n in (150, 7, 61)]
    seqs, worst = ex.generate(prompts, 6)
    assert [len(s) for s in seqs] == [156, 13, 67]
    assert worst <= 7 * 3 * 2.0 ** -8


def test_gradients_through_norm_rotation_and_aggregation():
    """Against float64 autograd of the formulas on the same inputs.  The chain rounds its
    intermediates (rotated q and k, gbar, E, the pair gradients, dq and dk of the aggregation)
    to bf16: six roundings, 2^-8 each, on the scale of each gradient's root mean square times
    its spread (element-wise errors are compared in the 2-norm)."""
    import generate_tango as ex
    r = ex.train_step(T=90)
    H, dh, mh, T = ex.H, ex.D_H, ex.M_H, 90
    lv = {n: r[n][0].double().cpu().requires_grad_() for n in ("q", "k", "g", "v")}
    gains = [x.double().cpu().requires_grad_() for x in r["gain"]]
    freqs = 10000.0 ** (-torch.arange(0, dh, 2, dtype=torch.float64) / dh)
    ang = torch.arange(T, dtype=torch.float64)[:, None, None] * freqs
    c, s = ang.cos(), ang.sin()

    def rope(x, gain):
        x = x.view(T, H, dh)
        z = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * gain
        a, b = z[..., :dh // 2], z[..., dh // 2:]
        z = torch.cat([a * c - b * s, a * s + b * c], -1)
        return z / z.norm(dim=-1, keepdim=True)  # the aggregation's own unit norm

    q, k = rope(lv["q"], gains[0]), rope(lv["k"], gains[1])
    w = torch.exp(10.0 * (torch.einsum("ihd,jhd->hij", q, k) - 1)).tril()
    gbar = torch.einsum("hij,jhc->ihc", w / w.sum(-1, keepdim=True), lv["g"].view(T, H, mh))
    (gbar * lv["v"].view(T, H, mh) * r["dout"][0].double().cpu().view(T, H, mh)).sum().backward()
    for got, want in ((r["dq"], lv["q"]), (r["dk"], lv["k"]), (r["dg"], lv["g"]), (r["dv"], lv["v"]),
                      (r["dgain"][0], gains[0]), (r["dgain"][1], gains[1])):
        got = got.double().cpu().reshape(want.shape)
        rel = ((got - want.grad).norm() / want.grad.norm()).item()
        assert rel <= 6 * 2.0 ** -8, rel
