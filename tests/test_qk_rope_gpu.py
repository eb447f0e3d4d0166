"""Norm and rotary position of q and k, their gradients, and the paged append, against the
formulas in float64.

Tolerances.  A stored value is off by its own rounding, half a step of its type (bf16
2^-8, fp32 2^-24, relative), plus the fp32 arithmetic: a head of d values is a sum of d
squares, a product with 1/|x|, a product with the gain and a rotation, each value then at
most (d/2 + 12) 2^-24 of the head's largest value off, and the angle (kept to 2^-25 turns)
another 2^-22 of it.  Gradients pass the same steps about twice and are compared on the
scale of the largest value of their head; gain gradients sum n of them in fp32, off by at
most (d + 12) 2^-23 of the sum of magnitudes with partial sums of at most 2^10 terms in turn.
"""
import math

import pytest
import torch

import cross_token_gated_gb300 as tg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _turn(z, pos, freqs, layout, sign=1.0):
    """z [N, H, d] float64, the first 2 len(freqs) columns turned by pos * freqs."""
    r = 2 * freqs.numel()
    z = z.clone()
    if r == 0:
        return z
    ang = sign * pos.double()[:, None] * freqs.double()
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    i = torch.arange(r // 2)
    a, b = (i, i + r // 2) if layout == tg.TG_ROPE_HALF else (2 * i, 2 * i + 1)
    x, y = z[..., a].clone(), z[..., b].clone()
    z[..., a], z[..., b] = x * c - y * s, x * s + y * c
    return z


def _scale(x, norm, eps):
    if norm == tg.TG_NORM_UNIT:
        return 1 / x.norm(dim=-1, keepdim=True).clamp(min=1e-12)
    if norm == tg.TG_NORM_RMS:
        return 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    return torch.ones_like(x[..., :1])


def _forward64(x, d_h, pos, freqs, layout, norm, gain, eps=1e-6):
    x = x.double().cpu().reshape(x.shape[0], -1, d_h)
    z = x * _scale(x, norm, eps) * (1.0 if gain is None else gain.double().cpu())
    return _turn(z, pos.cpu(), freqs.cpu(), layout)


def _close(got, want, dtype, d_h, times=1.0, what=""):
    """Element-wise: half a step of the value, plus the arithmetic's share of the head's scale."""
    got = got.double().cpu().reshape(want.shape)
    head = want.abs().amax(-1, keepdim=True)
    tol = HALF_STEP[dtype] * want.abs() * 1.001 + times * ((d_h / 2 + 12) * 2.0 ** -24 + 2.0 ** -22) * head + 1e-30
    worst = ((got - want).abs() / tol).max().item() if want.numel() else 0.0
    assert worst <= 1.0, (what, worst)


def _case(seed, rows, H, Hk, d_h, rotary, dtype, gains, far=1 << 20, fused=False):
    g = torch.Generator().manual_seed(seed)
    n = (H + Hk) * d_h
    x = torch.randn(rows, n + (8 if fused else 0), generator=g).to(DT[dtype]).cuda()
    if fused:  # column slices of one wider tensor
        q, k = x[:, 8:8 + H * d_h], x[:, 8 + H * d_h:]
    else:
        q, k = x[:, :H * d_h].contiguous(), x[:, H * d_h:].contiguous()
    pos = torch.randint(-5, far, (rows,), generator=g, dtype=torch.int32).cuda()
    freqs = tg.tg_rope_freqs(rotary) if rotary else None
    qg = (1 + 0.3 * torch.randn(d_h, generator=g)).cuda() if gains else None
    kg = (1 + 0.3 * torch.randn(d_h, generator=g)).cuda() if gains else None
    return q, (k if Hk else None), pos, freqs, qg, kg, g


SHAPES = [  # rows, H, Hk, d_h, rotary, layout, norm, gains, fused
    (1, 2, 2, 64, 64, 0, 1, False, False),
    (7, 2, 2, 64, 64, 1, 1, False, True),
    (1000, 16, 16, 32, 32, 0, 1, False, True),
    (333, 8, 2, 64, 32, 1, 2, True, False),
    (129, 3, 1, 128, 96, 0, 2, True, False),
    (50, 2, 0, 16, 16, 0, 1, False, False),
    (65, 2, 3, 64, 38, 0, 2, True, False),     # pairs that do not fill 16-byte vectors
    (31, 5, 5, 50, 50, 1, 1, True, False),     # a head of no whole vectors
    (9, 1, 1, 7, 6, 0, 2, True, False),        # an odd head width
    (40, 2, 2, 64, 0, 0, 0, True, False),      # no rotation, no norm
    (2500, 2, 2, 64, 64, 0, 2, True, False),   # several steps of a block
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=[str(s[0]) + "x" + str(s[3]) for s in SHAPES])
def test_forward(shape, dtype):
    rows, H, Hk, d_h, rotary, layout, norm, gains, fused = shape
    q, k, pos, freqs, qg, kg, _ = _case(1, rows, H, Hk, d_h, rotary, dtype, gains, fused=fused)
    fr = freqs if freqs is not None else torch.zeros(0, dtype=torch.float64)
    qo = torch.full((rows, H * d_h), float("nan"), dtype=DT[dtype], device="cuda")
    ko = torch.full((rows, Hk * d_h), float("nan"), dtype=DT[dtype], device="cuda") if Hk else None
    tg.tango_qk_norm_rope(q, k, qo, ko, freqs, H=H, H_k=Hk, positions=pos, layout=layout, norm=norm, q_gain=qg, k_gain=kg)
    _close(qo, _forward64(q, d_h, pos, fr, layout, norm, qg), dtype, d_h, what="q")
    if Hk:
        _close(ko, _forward64(k, d_h, pos, fr, layout, norm, kg), dtype, d_h, what="k")


def test_implicit_positions_and_in_place():
    """Without positions a row stands at its index along T; outputs may be the inputs."""
    g = torch.Generator().manual_seed(3)
    q = torch.randn(3, 37, 128, generator=g).cuda()
    k = torch.randn(3, 37, 128, generator=g).cuda()
    fr = tg.tg_rope_freqs(64)
    pos = torch.arange(37).repeat(3)
    want = [_forward64(t.reshape(-1, 128), 64, pos, fr, 0, 1, None) for t in (q, k)]
    tg.tango_qk_norm_rope(q, k, q, k, fr, H=2)
    _close(q, want[0], "f32", 64)
    _close(k, want[1], "f32", 64)


def test_agrees_with_the_block():
    """Unit norm and half layout from raw projections give the unit q, k that the block
    forms inside its projection (both round once to bf16: one step apart at most)."""
    g = torch.Generator().manual_seed(4)
    B, T, d, H, d_h, m = 2, 70, 64, 2, 64, 256
    h = torch.randn(B, T, d, generator=g).bfloat16().cuda()
    w = {n: (torch.randn(o, i, generator=g) / math.sqrt(i)).bfloat16().cuda()
         for n, o, i in (("Wq", H * d_h, d), ("Wk", H * d_h, d), ("Wg", m, d), ("Wv", m, d), ("Wo", d, m))}
    w["gamma"] = torch.ones(d).bfloat16().cuda()
    ws = tg.block_workspace(B, T, d, H, H * d_h, m, dtype=tg.TG_BF16)
    tg.tango_block_forward(h, w, torch.empty_like(h), H=H, ws=ws)
    off = -ws.data_ptr() % 256
    a256 = lambda x: (x + 255) // 256 * 256  # noqa: E731
    n = B * T * H * d_h * 2
    at = off + a256(B * T * d * 2)
    q_blk = ws[at:at + n].view(torch.bfloat16).reshape(B, T, -1)
    x = ws[off:off + B * T * d * 2].view(torch.bfloat16).reshape(B, T, d)
    raw = (x.float() @ w["Wq"].float().T)
    q = torch.empty_like(raw)
    tg.tango_qk_norm_rope(raw, None, q, None, tg.tg_rope_freqs(d_h), H=H)
    assert (q - q_blk.float()).abs().max().item() <= 2.0 ** -8 + 2.0 ** -12


def _backward64(x, dy, d_h, pos, freqs, layout, norm, gain, eps=1e-6):
    x = x.double().cpu().reshape(x.shape[0], -1, d_h)
    dy = dy.double().cpu().reshape(x.shape)
    r = _scale(x, norm, eps)
    n = x * r
    dz = _turn(dy, pos.cpu(), freqs.cpu(), layout, -1.0)
    dgain = (dz * n).sum((0, 1))
    mag = (dz * n).abs().sum((0, 1))
    dn = dz * (1.0 if gain is None else gain.double().cpu())
    if norm == tg.TG_NORM_NONE:
        return dn, dgain, mag, dn
    along = (n * dn).sum(-1, keepdim=True) / (1 if norm == tg.TG_NORM_UNIT else d_h)
    return r * (dn - n * along), dgain, mag, r * dn


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=[str(s[0]) + "x" + str(s[3]) for s in SHAPES])
def test_backward(shape, dtype):
    rows, H, Hk, d_h, rotary, layout, norm, gains, fused = shape
    q, k, pos, freqs, qg, kg, g = _case(2, rows, H, Hk, d_h, rotary, dtype, gains, fused=fused)
    fr = freqs if freqs is not None else torch.zeros(0, dtype=torch.float64)
    dqo = torch.randn(rows, H * d_h, generator=g).to(DT[dtype]).cuda()
    dko = torch.randn(rows, Hk * d_h, generator=g).to(DT[dtype]).cuda() if Hk else None
    dq, dk = torch.empty_like(dqo), torch.empty_like(dko) if Hk else None
    dqg, dkg = (torch.empty(d_h, device="cuda") if gains and x is not None else None for x in (q, k))
    kw = dict(H=H, H_k=Hk, positions=pos, layout=layout, norm=norm, q_gain=qg, k_gain=kg)
    tg.tango_qk_norm_rope_backward(q, k, dqo, dko, dq, dk, freqs, dq_gain=dqg, dk_gain=dkg, **kw)
    for x, dy, dx, gain, dgain in ((q, dqo, dq, qg, dqg), (k, dko, dk, kg, dkg)):
        if x is None:
            continue
        want, wg, mag, before = _backward64(x, dy, d_h, pos, fr, layout, norm, gain)
        got = dx.double().cpu().reshape(want.shape)
        scale = before.abs().amax(-1, keepdim=True) * 2
        tol = HALF_STEP[dtype] * want.abs() * 1.001 + 3 * ((d_h + 12) * 2.0 ** -24 + 2.0 ** -22) * scale + 1e-30
        assert ((got - want).abs() / tol).max().item() <= 1.0
        if dgain is not None:
            tol = ((d_h + 12) * 2.0 ** -23 + 2.0 ** -14) * mag + 1e-30
            assert ((dgain.double().cpu() - wg).abs() / tol).max().item() <= 1.0


def test_backward_against_differences():
    """The gradient of sum(dout * out) against central differences of the float64 formula,
    and of the fp32 kernel against it."""
    rows, H, d_h, rotary = 3, 2, 16, 12
    g = torch.Generator().manual_seed(9)
    x = torch.randn(rows, H * d_h, generator=g)
    dy = torch.randn(rows, H * d_h, generator=g)
    gain = 1 + 0.2 * torch.randn(d_h, generator=g)
    pos = torch.tensor([0, 5, 100000], dtype=torch.int32)
    fr = tg.tg_rope_freqs(rotary, device="cpu")
    for norm in (tg.TG_NORM_UNIT, tg.TG_NORM_RMS):
        def loss(t):
            return (_forward64(t, d_h, pos, fr, 1, norm, gain).reshape(rows, -1) * dy.double()).sum().item()
        num = torch.zeros(rows, H * d_h, dtype=torch.float64)
        for i in range(rows):
            for c in range(H * d_h):
                e = torch.zeros(rows, H * d_h, dtype=torch.float64)
                e[i, c] = 1e-5
                num[i, c] = (loss(x.double() + e) - loss(x.double() - e)) / 2e-5
        dx = torch.empty(rows, H * d_h, device="cuda")
        tg.tango_qk_norm_rope_backward(x.cuda(), None, dy.cuda(), None, dx, None, fr.cuda(), H=H, positions=pos.cuda(),
                                       layout=tg.TG_ROPE_INTERLEAVED, norm=norm, q_gain=gain.cuda())
        # differences: 1e-10 truncation, 1e-11 cancellation; the kernel: a few 1e-6 of the scale
        assert (dx.double().cpu() - num).abs().max().item() <= 2e-5 * num.abs().max().item()


def test_zero_vectors_and_empty():
    z = torch.zeros(2, 128, device="cuda")
    o, fr = torch.full_like(z, 7.0), tg.tg_rope_freqs(64)
    tg.tango_qk_norm_rope(z, None, o, None, fr, H=2)
    assert (o == 0).all()
    dy, dx = torch.ones_like(z), torch.empty_like(z)
    tg.tango_qk_norm_rope_backward(z, None, dy, None, dx, None, None, H=2)
    assert torch.allclose(dx, torch.full_like(dx, 1e12), rtol=1e-6)   # dn / 1e-12
    e = torch.zeros(0, 128, device="cuda")
    gain, dgain = torch.ones(64, device="cuda"), torch.full((64,), 3.0, device="cuda")
    tg.tango_qk_norm_rope(e, None, e, None, fr, H=2)
    tg.tango_qk_norm_rope_backward(e, None, e, None, e, None, fr, H=2, q_gain=gain, dq_gain=dgain)
    assert (dgain == 0).all()


def test_backward_repeats_bit_for_bit():
    q, k, pos, fr, qg, kg, g = _case(5, 5000, 8, 2, 64, 64, "bf16", True)
    dqo, dko = torch.randn(5000, 512, generator=g).bfloat16().cuda(), torch.randn(5000, 128, generator=g).bfloat16().cuda()
    outs = []
    for _ in range(3):
        r = [torch.empty_like(dqo), torch.empty_like(dko), torch.empty(64, device="cuda"), torch.empty(64, device="cuda")]
        tg.tango_qk_norm_rope_backward(q, k, dqo, dko, r[0], r[1], fr, H=8, H_k=2, positions=pos, norm=tg.TG_NORM_RMS,
                                       q_gain=qg, k_gain=kg, dq_gain=r[2], dk_gain=r[3])
        outs.append(r)
    for r in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], r))


def test_side_stream_and_graph():
    q, k, pos, fr, *_ = _case(6, 300, 2, 2, 64, 64, "bf16", False)
    want = [torch.empty_like(q), torch.empty_like(k)]
    tg.tango_qk_norm_rope(q, k, *want, fr, H=2, positions=pos)
    got = [torch.zeros_like(q), torch.zeros_like(k)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        tg.tango_qk_norm_rope(q, k, *got, fr, H=2, positions=pos)
        s.synchronize()
        assert torch.equal(got[0], want[0])
        got[0].zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            tg.tango_qk_norm_rope(q, k, *got, fr, H=2, positions=pos)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", [tg.TG_NORM_UNIT, tg.TG_NORM_RMS])
@pytest.mark.parametrize("d_h,rotary,layout", [(64, 64, 0), (64, 32, 1), (50, 38, 0)])
def test_a_nan_or_infinity_stays_in_its_head_and_is_not_lost(d_h, rotary, layout, norm, dtype):
    """The norm of a head with a NaN is NaN, and so is every value of it; a head with an infinity
    gives zeros, and NaN where the infinity and its pair stood.  Other heads and rows are as
    without them.  Gradients of such heads are NaN."""
    rows, H = 6, 3
    q, _, pos, freqs, _, _, g = _case(11, rows, H, 0, d_h, rotary, dtype, False)
    q[1, d_h + 5], q[3, 2 * d_h + d_h - 1], q[4, 7] = math.nan, math.nan, math.inf
    out = torch.zeros(rows, H * d_h, dtype=DT[dtype], device="cuda")
    tg.tango_qk_norm_rope(q, None, out, None, freqs, H=H, positions=pos, layout=layout, norm=norm)
    want = _forward64(q, d_h, pos, freqs, layout, norm, None)
    got = out.double().cpu().reshape(want.shape)
    assert want[1, 1].isnan().all() and want[3, 2].isnan().all() and want[4, 0].isnan().sum() == (2 if rotary > 7 else 1)
    assert torch.equal(got.isnan(), want.isnan())
    keep = torch.nan_to_num(want, nan=0.0)
    _close(torch.nan_to_num(got, nan=0.0), keep, dtype, d_h)
    dy, dx = torch.randn(rows, H * d_h, generator=g).to(DT[dtype]).cuda(), torch.zeros_like(out)
    tg.tango_qk_norm_rope_backward(q, None, dy, None, dx, None, freqs, H=H, positions=pos, layout=layout, norm=norm)
    bad = torch.zeros(rows, H, dtype=torch.bool)
    bad[1, 1] = bad[3, 2] = bad[4, 0] = True
    assert torch.equal(dx.cpu().reshape(rows, H, d_h).isnan(), bad[..., None].expand(-1, -1, d_h))


@pytest.mark.parametrize("d_h", [64, 50])
def test_fp32_norms_round_each_step_once(d_h):
    """Heads with one value a: the sum of squares is exact, so that the quotient by d_h, the sum
    with eps, the root, its inverse and the product are five roundings in a known order (unit:
    the last two, the root of a square being exact), the same as of these operations in fp32."""
    a = torch.arange(1, 4097, dtype=torch.float32)
    x = torch.zeros(len(a), d_h)
    x[torch.arange(len(a)), torch.arange(len(a)) % d_h] = a
    out = torch.zeros(len(a), d_h, device="cuda")
    for norm, want in ((tg.TG_NORM_UNIT, a * (1 / a)), (tg.TG_NORM_RMS, a * (1 / (a * a / d_h + 1e-6).sqrt()))):
        tg.tango_qk_norm_rope(x.cuda(), None, out, None, None, H=1, norm=norm)
        assert torch.equal(out.cpu().sum(1), want)


@pytest.mark.parametrize("d_h", [64, 50])
def test_fp32_cosines_and_sines(d_h):
    """Pairs (1, 0) turn into the cosine and sine themselves: off by the angle, which fp32 holds to
    pi 2^-27 from the next quarter turn (and 64 bits of turns a position: 2^-30 at 2^24), and by one
    unit of sincospi, 2^-24 below 1."""
    rows = 20000
    g = torch.Generator().manual_seed(12)
    pos = torch.randint(-(1 << 24), 1 << 24, (rows,), generator=g, dtype=torch.int32)
    pos[:64] = torch.arange(64)
    freqs = tg.tg_rope_freqs(d_h, device="cpu")
    x = torch.zeros(rows, d_h)
    x[:, :d_h // 2] = 1
    out = torch.empty(rows, d_h, device="cuda")
    tg.tango_qk_norm_rope(x.cuda(), None, out, None, freqs.cuda(), H=1, positions=pos.cuda(), norm=tg.TG_NORM_NONE)
    # the angle in 64-bit turns, reduced exactly in integers
    frac = [int(f.item() / (2 * math.pi) % 1.0 * 2.0 ** 64) for f in freqs]
    ang = torch.tensor([[(f * p) % (1 << 64) / 2.0 ** 64 for f in frac] for p in pos.tolist()], dtype=torch.float64)
    want = torch.cat([(2 * math.pi * ang).cos(), (2 * math.pi * ang).sin()], 1)
    assert (out.double().cpu() - want).abs().max().item() <= math.pi * 2.0 ** -27 + 2.0 ** -24 + 2.0 ** -30
