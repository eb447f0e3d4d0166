"""Lookup, norm, distillation and sampling against plain 64-bit forms, at the sizes and masks where
they can go wrong.

Bounds: every sum of n terms in fp32, in any order, is off by at most n u sum|terms| with u = 2^-24;
stored results by half a step of their type, finfo.eps / 2 relative.  Each test counts those.
"""
import math

import pytest
import torch

import cross_token_gated_gb300 as tg

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32, I32, F64 = torch.bfloat16, torch.float32, torch.int32, torch.float64


def half_step(dt):
    return torch.finfo(dt).eps / 2


def normal(gen, *shape, dt=F32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def within(got, want, bound):
    got = got.double()
    assert torch.isfinite(got).all()
    worst = ((got - want).abs() / bound.clamp(min=1e-300)).max().item() if got.numel() else 0.0
    assert ((got - want).abs() <= bound).all(), f"{worst} of the bound"


def no_error():
    assert tg.tg_check_device_error() == (tg.TG_OK, 0)


def flagged(kernel):
    st, word = tg.tg_check_device_error()
    assert st == tg.TG_ERR_DEVICE and (word >> 8) & 255 == kernel


# ------------------------------------------------------------------------------ lookup

@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("rows,d,vocab", [(1, 1, 1), (7, 7, 5), (33, 64, 1000), (100, 513, 300), (4097, 512, 32768), (9, 2048, 40)])
@pytest.mark.parametrize("scale", [1.0, 22.627417])
def test_embed(lib, dt, rows, d, vocab, scale):
    gen = generator(rows + d)
    E = normal(gen, vocab, d, dt=dt)
    ids = torch.randint(0, vocab, (rows,), generator=gen, device="cuda", dtype=I32)
    ids[::3] = -1
    wide = torch.full((rows, d + 5), 7.0, dtype=dt, device="cuda")
    tg.tango_embed(ids, E, wide[:, :d], scale=scale)
    want = torch.where((ids < 0)[:, None], torch.zeros((), dtype=dt, device="cuda"),
                       (E.float() * scale).to(dt)[ids.clamp(min=0).long()])
    assert torch.equal(wide[:, :d], want) and (wide[:, d:] == 7).all()
    out = torch.empty(rows, d, dtype=dt, device="cuda")
    assert torch.equal(tg.tango_embed(ids, E, out, scale=scale), want)
    no_error()


def test_embed_pad_and_bad_ids(lib):
    E = normal(generator(0), 10, 16, dt=BF)
    out = torch.empty(4, 16, dtype=BF, device="cuda")
    tg.tango_embed(torch.tensor([3, 9, 3, 0], dtype=I32, device="cuda"), E, out, pad_id=3)
    assert torch.equal(out[1::2], E[[9, 0]]) and (out[::2] == 0).all()
    no_error()
    for bad in (10, -2, 2 ** 31 - 1, -2 ** 31):
        ids = torch.tensor([1, bad, 2, -1], dtype=I32, device="cuda")
        tg.tango_embed(ids, E, out)
        assert torch.equal(out[::2], E[[1, 2]]) and (out[1::2] == 0).all()
        flagged(4)
        dE = torch.empty(10, 16, device="cuda")
        tg.tango_embed_backward(ids, torch.ones(4, 16, dtype=BF, device="cuda"), dE)
        assert dE.sum() == 32 and (dE[1:3] == 1).all()
        flagged(4)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("d", [64, 7])
@pytest.mark.parametrize("scale", [math.inf, math.nan, -2.0])
def test_embed_padding_is_zero_at_any_scale(lib, dt, d, scale):
    """Rows without a token are zeros (+0) whatever the factor."""
    E = normal(generator(31), 10, d, dt=dt)
    ids = torch.tensor([-1, 4, -1], dtype=I32, device="cuda")
    out = torch.full((3, d), 5.0, dtype=dt, device="cuda")
    tg.tango_embed(ids, E, out, scale=scale)
    assert (out[::2].view(torch.int16 if dt is BF else I32) == 0).all()
    assert torch.equal(out[1].isnan(), (E[4].float() * scale).isnan())
    no_error()


def embed_ids(kind, rows, vocab, gen):
    if kind == "same":
        return torch.full((rows,), vocab // 2, dtype=I32, device="cuda")
    if kind == "pads":
        return torch.full((rows,), -1, dtype=I32, device="cuda")
    if kind == "few":  # three long lists at the ends and one in the middle
        return torch.tensor([0, vocab - 1, vocab // 3], dtype=I32, device="cuda")[torch.randint(0, 3, (rows,), generator=gen, device="cuda")]
    if kind == "zipf":
        u = torch.rand(rows, generator=gen, device="cuda")
        return (torch.exp(u * math.log(vocab)) - 1).to(I32).clamp(0, vocab - 1)
    ids = torch.randint(0, vocab, (rows,), generator=gen, device="cuda", dtype=I32)
    return torch.where(torch.rand(rows, generator=gen, device="cuda") < 0.2, torch.full_like(ids, -1), ids)


@pytest.mark.parametrize("rows,d,vocab,kind", [
    (1, 1, 1, "same"), (0, 8, 5, "mixed"), (31, 7, 3, "mixed"), (33, 64, 1000, "mixed"), (1000, 513, 70, "zipf"),
    (5003, 768, 32768, "zipf"), (16384, 512, 32768, "zipf"), (4097, 24, 250003, "mixed"), (3000, 128, 999, "pads"),
    (9001, 256, 999, "same"), (70001, 40, 1000, "same"), (20000, 1000, 50257, "few"), (40, 4096, 60, "few"),
])
@pytest.mark.parametrize("dt,gt", [(BF, F32), (F32, F32), (BF, BF)])
def test_embed_backward(lib, rows, d, vocab, kind, dt, gt):
    gen = generator(rows + d + vocab)
    ids = embed_ids(kind, rows, vocab, gen)
    dout = normal(gen, rows, d, dt=dt)
    base = normal(gen, vocab, d, dt=gt)
    scale, live = 1.7, ids >= 0
    want = torch.zeros(vocab, d, dtype=F64, device="cuda").index_add_(0, ids[live].long(), dout.double()[live])
    size = torch.zeros(vocab, d, dtype=F64, device="cuda").index_add_(0, ids[live].long(), dout.double().abs()[live])
    count = torch.zeros(vocab, 1, dtype=F64, device="cuda").index_add_(0, ids[live].long(), torch.ones(int(live.sum()), 1, dtype=F64, device="cuda"))
    for b in (None, base):
        dE = torch.full((vocab, d), math.nan, dtype=gt, device="cuda")
        tg.tango_embed_backward(ids, dout, dE, scale=scale, base=b)
        ref = want * scale + (0 if b is None else b.double())
        # the sum, the factor (also its own rounding from 1.7), the base's addition, the store
        bound = U * scale * size * (count + 3) + 2 * U * ref.abs() + half_step(gt) * ref.abs() * (1 + 2 ** -6)
        within(dE, ref, bound)
        again = torch.empty_like(dE) if b is None else b.clone()  # the same bits, also added in place
        tg.tango_embed_backward(ids, dout, again, scale=scale, base=None if b is None else again)
        assert torch.equal(dE, again)
    no_error()


def test_embed_backward_slices_pad_and_nan(lib):
    """Rows at a pitch, a pad id inside the vocabulary whose rows hold NaN, untouched memory."""
    gen = generator(3)
    wide = normal(gen, 500, 96, dt=BF)
    ids = torch.randint(0, 50, (500,), generator=gen, device="cuda", dtype=I32)
    dout = wide[:, 8:72]
    dout[ids == 7] = math.nan
    dE = torch.empty(50, 64, device="cuda")
    tg.tango_embed_backward(ids, dout, dE, pad_id=7)
    want = torch.zeros(50, 64, dtype=F64, device="cuda").index_add_(0, ids[ids != 7].long(), dout.double()[ids != 7])
    assert (dE[7] == 0).all()
    assert (dE.double() - want).abs().max() <= 500 * U * 100
    off = normal(gen, 500 * 63 + 1, dt=BF)[1:].view(500, 63)  # no row is aligned
    dE = torch.empty(50, 63, device="cuda")
    tg.tango_embed_backward(ids, off, dE)
    want = torch.zeros(50, 63, dtype=F64, device="cuda").index_add_(0, ids.long(), off.double())
    assert (dE.double() - want).abs().max() <= 500 * U * 100


# -------------------------------------------------------------------------------- norm

def norm_ref(x, gamma, beta, layer, eps):
    x = x.double()
    mu = x.mean(-1, keepdim=True) if layer else torch.zeros((), dtype=F64, device=x.device)
    r = 1 / ((x - mu).square().mean(-1, keepdim=True) + eps).sqrt()
    n = (x - mu) * r
    y = n if gamma is None else n * gamma.double()
    return y if beta is None else y + beta.double(), n, r


NORM_SHAPES = [(1, 1), (3, 7), (5, 64), (1, 512), (33, 512), (1000, 513), (4096, 512), (257, 768), (65, 1000), (17, 2048),
               (9, 4096), (7, 8192), (3, 16384), (2, 40000), (300, 24), (130, 4104)]


@pytest.mark.parametrize("rows,d", NORM_SHAPES)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("layer,affine", [(False, True), (True, True), (True, False)])
def test_norm(lib, rows, d, dt, layer, affine):
    gen = generator(rows * d)
    x = normal(gen, rows, d + 8, dt=dt, scale=1.5)[:, :d] if d % 3 else normal(gen, rows, d, dt=dt, scale=1.5)
    x += 0.5
    gamma = (1 + normal(gen, d, scale=0.3)).to(dt) if affine else None
    beta = normal(gen, d, dt=dt, scale=0.2) if affine and layer else None
    y = torch.empty(rows, d, dtype=dt, device="cuda")
    tg.tango_norm(x, gamma, beta, y, norm=tg.TG_NORM_LAYER if layer else tg.TG_NORM_RMS, eps=1e-5)
    want, n, r = norm_ref(x, gamma, beta, layer, 1e-5)
    g = 1.0 if gamma is None else gamma.double().abs()
    b = 0.0 if beta is None else beta.double().abs()
    k = d / 32 + 24  # terms of a thread and of the joins, and single roundings
    bound = k * U * (r * x.double().abs().mean(-1, keepdim=True) + n.abs()) * g + 2 * U * (want.abs() + b)
    within(y, want, bound + half_step(dt) * want.abs() * (1 + 2 ** -6))
    if x.is_contiguous():
        tg.tango_norm(x, gamma, beta, x, norm=tg.TG_NORM_LAYER if layer else tg.TG_NORM_RMS, eps=1e-5)
        assert torch.equal(x, y)


@pytest.mark.parametrize("rows,d", NORM_SHAPES)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("layer,affine,res", [(False, True, True), (True, True, False), (True, False, True), (False, False, False)])
def test_norm_backward(lib, rows, d, dt, layer, affine, res):
    gen = generator(rows * d + 1)
    x = normal(gen, rows, d + 8, dt=dt, scale=1.5)[:, :d] if d % 3 else normal(gen, rows, d, dt=dt, scale=1.5)
    x += 0.5
    gamma = (1 + normal(gen, d, scale=0.3)).to(dt) if affine else None
    dy, dres = normal(gen, rows, d, dt=dt), normal(gen, rows, d, dt=dt) if res else None
    dx = torch.empty(rows, d, dtype=dt, device="cuda")
    dg = torch.empty(d, device="cuda") if affine else None
    db = torch.empty(d, device="cuda") if layer else None
    how = dict(norm=tg.TG_NORM_LAYER if layer else tg.TG_NORM_RMS, eps=1e-5)
    tg.tango_norm_backward(x, gamma, dy, dx, dres=dres, dgamma=dg, dbeta=db, **how)
    _, n, r = norm_ref(x, None, None, layer, 1e-5)
    dn = dy.double() * (1.0 if gamma is None else gamma.double())
    m1 = (dn * n).mean(-1, keepdim=True)
    m0 = dn.mean(-1, keepdim=True) if layer else 0.0
    want = r * (dn - n * m1 - m0) + (dres.double() if res else 0.0)
    k = d / 32 + 24
    size = r * x.double().abs().mean(-1, keepdim=True) + n.abs()  # n is off by k U of this at most
    terms = 2 * dn.abs() + 2 * size * (dn.abs() * size).mean(-1, keepdim=True) * 2 + 2 * dn.abs().mean(-1, keepdim=True)
    bound = k * U * r * terms + 2 * U * (want.abs() + (dres.double().abs() if res else 0.0))
    within(dx, want, bound + half_step(dt) * want.abs() * (1 + 2 ** -6))
    if affine:
        within(dg, (dy.double() * n).sum(0), (rows + 2 * k) * U * (dy.double().abs() * size).sum(0))
    if layer:
        within(db, dy.double().sum(0), rows * U * dy.double().abs().sum(0))
    # in place over dy, and over the residual's gradient: the same bits
    over = dy.clone()
    dg2 = None if dg is None else torch.empty_like(dg)
    tg.tango_norm_backward(x, gamma, over, over, dres=dres, dgamma=dg2, dbeta=db, **how)
    assert torch.equal(over, dx) and (dg is None or torch.equal(dg, dg2))
    if res:
        over = dres.clone()
        tg.tango_norm_backward(x, gamma, dy, over, dres=over, **how)
        assert torch.equal(over, dx)


@pytest.mark.parametrize("rows,d", [(700, 4096), (400, 16384), (900, 8191), (1500, 16392), (1300, 40000)])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("layer", [False, True])
def test_norm_several_wide_rows_of_a_block(lib, rows, d, dt, layer):
    """More rows than blocks where many threads share a row: the next row is on its way, buffers are
    taken in turn and the weights' gradients are summed over a block's rows."""
    gen = generator(rows + d)
    x = normal(gen, rows, d, dt=dt, scale=1.5) + 0.5
    gamma, dy = (1 + normal(gen, d, scale=0.3)).to(dt), normal(gen, rows, d, dt=dt)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dg, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    how = dict(norm=tg.TG_NORM_LAYER if layer else tg.TG_NORM_RMS, eps=1e-5)
    tg.tango_norm(x, gamma, None, y, **how)
    tg.tango_norm_backward(x, gamma, dy, dx, dgamma=dg, dbeta=db, **how)
    want, n, r = norm_ref(x, gamma, None, layer, 1e-5)
    k = d / 32 + 24  # terms of a thread and of the joins, and single roundings
    size = r * x.double().abs().mean(-1, keepdim=True) + n.abs()  # n is off by k U of this at most
    within(y, want, k * U * size * gamma.double().abs() + 2 * U * want.abs() + half_step(dt) * want.abs() * (1 + 2 ** -6))
    dn = dy.double() * gamma.double()
    want = r * (dn - n * (dn * n).mean(-1, keepdim=True) - (dn.mean(-1, keepdim=True) if layer else 0.0))
    terms = 2 * dn.abs() + 4 * size * (dn.abs() * size).mean(-1, keepdim=True) + 2 * dn.abs().mean(-1, keepdim=True)
    within(dx, want, k * U * r * terms + 2 * U * want.abs() + half_step(dt) * want.abs() * (1 + 2 ** -6))
    within(dg, (dy.double() * n).sum(0), (rows + 2 * k) * U * (dy.double().abs() * size).sum(0))
    within(db, dy.double().sum(0), rows * U * dy.double().abs().sum(0))


def test_norm_backward_by_differences(lib):
    """fp32 gradients of a scalar against its differences along one direction."""
    gen = generator(9)
    x, dy, v = (normal(gen, 6, 50) for _ in range(3))
    gamma = 1 + normal(gen, 50, scale=0.3)
    for layer in (False, True):
        how = dict(norm=tg.TG_NORM_LAYER if layer else tg.TG_NORM_RMS, eps=1e-5)
        dx, dg = torch.empty_like(x), torch.empty(50, device="cuda")
        tg.tango_norm_backward(x, gamma, dy, dx, dgamma=dg, **how)

        def loss(xx, gg):
            return (norm_ref(xx, gg, None, layer, 1e-5)[0] * dy.double()).sum()
        h = 1e-5
        d = (loss(x.double() + h * v.double(), gamma) - loss(x.double() - h * v.double(), gamma)) / (2 * h)
        # the difference's own error is about h^2 and 1e-16 / h; the gradient's is fp32
        assert abs((dx.double() * v).sum() - d) <= 1e-4 * (dx.double() * v).abs().sum()
        d = (loss(x, gamma.double() + h * v[0].double()) - loss(x, gamma.double() - h * v[0].double())) / (2 * h)
        assert abs((dg.double() * v[0]).sum() - d) <= 1e-4 * (dg.double() * v[0]).abs().sum()


@pytest.mark.parametrize("dt,d", [(F32, 6128), (F32, 6132), (F32, 6144), (F32, 6148), (BF, 12256), (BF, 12264), (BF, 12288),
                                  (BF, 12296), (F32, 8192), (F32, 8191), (F32, 6143), (F32, 6147), (BF, 16384), (BF, 8191)])
def test_norm_widths_about_48_kb_of_weights(lib, dt, d):
    """Gain and bias in shared memory, up to and past what a kernel may have without asking."""
    gen = generator(d)
    x, gamma, beta = normal(gen, 3, d, dt=dt), normal(gen, d, dt=dt), normal(gen, d, dt=dt)
    y = torch.empty_like(x)
    for layer in (False, True):
        tg.tango_norm(x, gamma, beta, y, norm=tg.TG_NORM_LAYER if layer else tg.TG_NORM_RMS, eps=1e-5)
        want, n, r = norm_ref(x, gamma, beta, layer, 1e-5)
        size = r * x.double().abs().mean(-1, keepdim=True) + n.abs()
        bound = (d / 32 + 24) * U * size * gamma.double().abs() + 2 * U * (want.abs() + beta.double().abs())
        within(y, want, bound + half_step(dt) * want.abs() * (1 + 2 ** -6))


def test_norm_special_rows(lib):
    """Zero rows stay finite, a NaN stays in its row, rows of one value, an empty batch."""
    x = torch.zeros(4, 64, dtype=BF, device="cuda")
    x[1, 5], x[2] = math.nan, 3.0
    y = torch.empty_like(x)
    for norm in (tg.TG_NORM_RMS, tg.TG_NORM_LAYER):
        tg.tango_norm(x, None, None, y, norm=norm)
        assert (y[0] == 0).all() and y[1].isnan().all() and (y[3] == 0).all()
        assert (y[2] == (0 if norm == tg.TG_NORM_LAYER else 1)).all()
    dg, db = torch.full((64,), 5.0, device="cuda"), torch.full((64,), 5.0, device="cuda")
    tg.tango_norm_backward(x[:0], y[0], y[:0], y[:0], norm=tg.TG_NORM_LAYER, dgamma=dg, dbeta=db)
    assert (dg == 0).all() and (db == 0).all()


# ------------------------------------------------------------------------- distillation

def distill_ref(z, t, ids, T):
    """(loss, q, target), all in 64 bits; absent entries are -1 or -inf."""
    V = z.shape[-1]
    live = (ids >= 0) & (ids < V) & (t != -math.inf)
    some = live.any(-1)
    tl = torch.where(live, t.double(), torch.full((), -math.inf, dtype=F64, device=z.device)) / T
    logp = torch.where(some[:, None], torch.log_softmax(tl, -1), -math.inf)
    p = logp.exp()
    logq = torch.log_softmax(z.double() / T, -1)
    at = ids.clamp(0, V - 1).long()
    terms = torch.where(p > 0, p * (logp - logq.gather(1, at)), 0.0)
    loss = T * T * terms.sum(-1)
    target = torch.zeros_like(logq).scatter_add_(1, at, p)
    return torch.where(some, loss, 0.0), torch.where(some[:, None], logq.exp(), 0.0), target, logp, logq.gather(1, at), p


def distill_inputs(gen, rows, V, K, dt, scale=2.5):
    z = normal(gen, rows, V, dt=dt, scale=scale)
    v, i = (z.float() + normal(gen, rows, V)).topk(K, dim=1)
    return z, v.contiguous(), i.to(I32)


def check_distill(z, t, ids, T, dloss, loss, dz):
    want, q, target, logp, logq, p = distill_ref(z, t, ids, T)
    V, K = z.shape[-1], ids.shape[-1]
    # exponents y = (z - max) / T carry 2 roundings, the exponential 2^-22, the sum V / 512 + 16 terms
    reach = ((z.double().amax(-1, keepdim=True) - z.double()) / T).clamp(max=90.0)
    rel = U * (3 * reach + 8 + V / 256 + 40)
    t_reach = torch.where(p > 0, (t.amax(-1, keepdim=True) - t).double() / T, 0.0)
    rel_p = U * (3 * t_reach + 8 + K / 16 + 20)
    if loss is not None:
        a = torch.where(p > 0, logp.abs() + logq.abs(), 0.0)
        z_at = rel.gather(1, ids.clamp(0, V - 1).long())
        bound = T * T * (torch.where(p > 0, p * (a * (rel_p + (K / 16 + 20) * U) + rel_p + z_at + 8 * U * (a + 1)), 0.0)).sum(-1)
        within(loss, want, bound)
    if dz is not None:
        f = (dloss.double() * T)[:, None]
        ref = f * (q - target)
        tb = torch.zeros_like(q).scatter_add_(1, ids.clamp(0, V - 1).long(), torch.where(p > 0, p * (rel_p + K * U), 0.0))
        bound = f.abs() * (q * rel + tb + 2 * U * (q + target)) + 3 * U * ref.abs() + half_step(z.dtype) * ref.abs() * (1 + 2 ** -6)
        within(dz, ref, bound + 2.0 ** -133)  # the smallest steps of both types are denormal


@pytest.mark.parametrize("rows,V,K", [(1, 1, 1), (3, 5, 2), (7, 33, 33), (5, 1000, 1), (300, 1003, 17), (65, 32768, 64),
                                      (9, 32771, 100), (4, 50257, 256), (2, 131072, 1024), (3, 200000, 8), (620, 64, 5)])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T", [1.0, 2.0, 0.7])
def test_distill(lib, rows, V, K, dt, T):
    gen = generator(rows + V + K)
    z, t, ids = distill_inputs(gen, rows, V, K, dt)
    ids[1::4] = -1                      # padded rows
    if K > 2:
        ids[0, 1] = -1                  # an absent entry
        t[-1, 0] = -math.inf            # another, by its logit
        ids[-1, 2] = ids[-1, 1]         # the same token twice
    dloss = normal(gen, rows)
    loss, stats = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    tg.tango_distill(z, t, ids, loss, temperature=T, stats=stats)
    check_distill(z, t, ids, T, None, loss, None)
    dz = torch.full_like(z, math.nan)
    tg.tango_distill_backward(z, t, ids, dloss, dz, temperature=T, stats=stats)
    check_distill(z, t, ids, T, dloss, None, dz)
    one, both = torch.full_like(z, math.nan), torch.empty_like(loss)
    tg.tango_distill_backward(z, t, ids, dloss, one, temperature=T, loss=both)
    check_distill(z, t, ids, T, dloss, both, one)
    assert (dz[1::4] == 0).all() and (one[1::4] == 0).all() and (loss[1::4] == 0).all()
    over = z.clone()                    # in place
    tg.tango_distill_backward(over, t, ids, dloss, over, temperature=T)
    assert torch.equal(over, one)
    no_error()


@pytest.mark.parametrize("rows,V,K", [(4001, 203, 12), (1500, 9000, 40), (1001, 40009, 5)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_distill_many_rows(lib, rows, V, K, dt):
    """Several rows for every block, with padding in runs and alone, repeated and absent entries."""
    gen = generator(rows)
    z, t, ids = distill_inputs(gen, rows, V, K, dt)
    some = torch.randint(0, K, (rows, 3), generator=gen, device="cuda")
    ids.scatter_(1, some, ids.gather(1, some.flip(1)))                   # repeated tokens
    ids[torch.rand(rows, K, generator=gen, device="cuda") < 0.1] = -1
    ids[torch.rand(rows, generator=gen, device="cuda") < 0.3] = -1       # padding
    ids[rows // 3: rows // 3 + 900] = -1
    dloss, loss, stats = normal(gen, rows), torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    tg.tango_distill(z, t, ids, loss, temperature=1.5, stats=stats)
    check_distill(z, t, ids, 1.5, None, loss, None)
    dz, one = torch.full_like(z, math.nan), torch.full_like(z, math.nan)
    tg.tango_distill_backward(z, t, ids, dloss, dz, temperature=1.5, stats=stats)
    check_distill(z, t, ids, 1.5, dloss, None, dz)
    both = torch.empty_like(loss)
    tg.tango_distill_backward(z, t, ids, dloss, one, temperature=1.5, loss=both)
    check_distill(z, t, ids, 1.5, dloss, both, one)
    no_error()


@pytest.mark.parametrize("dt", [BF, F32])
def test_distill_pitches(lib, dt):
    """Rows of a padded vocabulary, aligned or not: what lies between them is neither read nor written."""
    gen = generator(5)
    for V, pitch, first in ((1000, 1024, 0), (1001, 1003, 1), (32768, 32776, 0)):
        z, t, ids = distill_inputs(gen, 6, V, 9, dt)
        wide = torch.full((6, pitch), math.nan, dtype=dt, device="cuda")
        wide[:, first:first + V] = z
        out = torch.full((6, pitch + 8), 3.0, dtype=dt, device="cuda")
        dloss = normal(gen, 6)
        loss = torch.empty(6, device="cuda")
        tg.tango_distill_backward(wide[:, first:first + V], t, ids, dloss, out[:, first:first + V], loss=loss)
        check_distill(z, t, ids, 1.0, dloss, loss, out[:, first:first + V].contiguous())
        assert (out[:, first + V:] == 3).all() and (out[:, :first] == 3).all()


@pytest.mark.parametrize("dt", [BF, F32])
def test_distill_masked_and_extreme_logits(lib, dt):
    gen = generator(6)
    low = torch.finfo(dt).min
    z, t, ids = distill_inputs(gen, 8, 777, 4, dt)
    free = torch.ones(777, dtype=torch.bool, device="cuda")
    free[ids.long().flatten()] = False
    z[:, free.nonzero()[:300, 0]] = -math.inf    # masked tokens without entries
    z[1, free] = low                             # the type's lowest value
    z[2] = low                                   # a whole row of it: uniform
    z[3] = -math.inf                             # nothing above -inf: q = 0
    z[4, ids[4, 0].long()] = -math.inf           # an entry on a masked token
    z[5, 3] = math.nan
    ids[6] = 777                                 # outside of the vocabulary
    t[7] = -math.inf                             # no entry left
    dloss = torch.ones(8, device="cuda")
    loss, both, dz, one = torch.empty(8, device="cuda"), torch.empty(8, device="cuda"), torch.empty_like(z), torch.empty_like(z)
    stats = torch.empty(8, 2, device="cuda")
    tg.tango_distill(z, t, ids, loss, stats=stats)
    flagged(7)
    tg.tango_distill_backward(z, t, ids, dloss, dz, stats=stats)
    flagged(7)
    tg.tango_distill_backward(z, t, ids, dloss, one, loss=both)
    flagged(7)
    for l, g in ((loss, dz), (both, one)):
        rows = [0, 1, 2]
        check_distill(z[rows], t[rows], ids[rows], 1.0, dloss[rows], l[rows], g[rows])
        assert l[3] == math.inf and l[4] == math.inf
        p = torch.softmax(t[3].double(), -1)
        want = torch.zeros(777, dtype=F64, device="cuda").scatter_add_(0, ids[3].long(), -p)
        within(g[3], want, (half_step(dt) * 1.02 + 60 * U) * want.abs())
        assert torch.isfinite(g[4]).all() and abs(g[4].double().sum().item()) <= 777 * half_step(dt)
        assert l[5].isnan() and g[5].isnan().all()
        assert l[6] == 0 and l[7] == 0 and (g[6:] == 0).all()


@pytest.mark.parametrize("V", [777, 40000])
@pytest.mark.parametrize("dt", [F32, BF], ids=["fp32", "bf16"])
def test_distill_infinite_logits(lib, dt, V):
    # +inf: softmax has inf - inf.  A student's reaches the whole row, a teacher's its entries' columns.
    gen = generator(9)
    z, t, ids = distill_inputs(gen, 3, V, 5, dt)
    ids[:] = torch.tensor([0, 5, 9, V // 2, V - 1], device="cuda", dtype=I32)
    want_z, want_t = z[2:].clone(), t[2:].clone()
    z[0, 3], t[1, 2] = math.inf, math.inf
    loss, dz = torch.empty(3, device="cuda"), torch.empty_like(z)
    tg.tango_distill_backward(z, t, ids, torch.ones(3, device="cuda"), dz, loss=loss)
    assert loss[:2].isnan().all() and dz[0].isnan().all()
    entries = torch.zeros(V, dtype=torch.bool, device="cuda")
    entries[ids[1].long()] = True
    assert dz[1, entries].isnan().all() and torch.isfinite(dz[1, ~entries]).all()
    # The finite row is held to the bounds on sums, not to its bits alone: row 2 of 777 bf16 values starts
    # 3,108 = 194 * 16 + 4 bytes in, so its vectors, and with them the order of its sums, are others.
    check_distill(want_z, want_t, ids[2:], 1.0, torch.ones(1, device="cuda"), loss[2:], dz[2:])


def test_distill_is_cross_entropy_with_one_entry(lib):
    gen = generator(8)
    z = normal(gen, 50, 999, scale=3.0)
    label = torch.randint(0, 999, (50, 1), generator=gen, device="cuda", dtype=I32)
    loss = torch.empty(50, device="cuda")
    tg.tango_distill(z, normal(gen, 50, 1), label, loss)
    want = torch.nn.functional.cross_entropy(z.double(), label[:, 0].long(), reduction="none")
    within(loss, want, U * 100 * (want.abs() + 10))


def test_distill_gradient_by_differences(lib):
    gen = generator(10)
    z, t, ids = distill_inputs(gen, 4, 60, 5, F32)
    v = normal(gen, 4, 60).double()
    dloss, dz, h = normal(gen, 4), torch.empty_like(z), 1e-5
    tg.tango_distill_backward(z, t, ids, dloss, dz, temperature=1.5)

    def total(zz):
        return (distill_ref(zz, t, ids, 1.5)[0] * dloss.double()).sum()
    d = (total(z.double() + h * v) - total(z.double() - h * v)) / (2 * h)
    assert abs((dz.double() * v).sum() - d) <= 1e-4 * (dz.double() * v).abs().sum()


# ---------------------------------------------------------------------------- sampling

def sample_ref(x, u, T, k, p, m):
    """Tokens and logprobs by the definition, row by row in 64 bits on the host."""
    import numpy as np
    x = x.double().cpu().numpy().copy()
    x[np.isnan(x)] = -np.inf
    f = [np.broadcast_to(np.asarray(s.double().cpu() if torch.is_tensor(s) else np.float64(np.float32(s))), (len(x),)) for s in (u, T, k, p, m)]
    tok, lp = [], []
    for row, uu, TT, kk, pp, mm in zip(x, *f):
        top = row.max()
        if top == -np.inf:
            tok.append(-1), lp.append(-math.inf)
            continue
        if TT == 0:
            tok.append(int(row.argmax())), lp.append(0.0)
            continue
        with np.errstate(invalid="ignore"):
            w = np.where(row == top, 1.0, np.exp(np.where(row == top, 0.0, row - top) / TT))
        w[~(w >= 2.0 ** -40)] = 0
        order = np.lexsort((np.arange(len(row)), -row))
        order = order[w[order] > 0]
        if kk > 0:
            order = order[:int(kk)]
        s = w[order]
        n = len(s)
        if pp < 1:
            before = np.cumsum(s) - s
            n = max(1, int((before < pp * math.fsum(s)).sum()))
        n = max(1, min(n, int((s >= mm).sum())))
        kept = np.sort(order[:n])
        c = np.cumsum(w[kept])
        j = min(n - 1, int((c <= uu * c[-1]).sum()))
        tok.append(int(kept[j])), lp.append(math.log(w[kept[j]] / c[-1]))
    return torch.tensor(tok, dtype=I32, device="cuda"), torch.tensor(lp, dtype=F64, device="cuda")


def check_sample(x, u, T=1.0, k=0, p=1.0, m=0.0):
    token = torch.full((x.shape[0],), -7, dtype=I32, device="cuda")
    logprob = torch.empty(x.shape[0], device="cuda")
    tg.tango_sample(x, u, token, temperature=T, top_k=k, top_p=p, min_p=m, logprob=logprob)
    want, lp = sample_ref(x, u, T, k, p, m)
    assert torch.equal(token, want), (token[token != want], want[token != want])
    live = torch.isfinite(lp)
    assert torch.equal(torch.isfinite(logprob), live)
    # the ratio is rounded three times, the logarithm to 2 units of its last place
    within(logprob[live], lp[live], (4 * U + 4 * U * lp.abs())[live])
    only = torch.empty_like(token)
    tg.tango_sample(x, u, only, temperature=T, top_k=k, top_p=p, min_p=m)
    assert torch.equal(only, token)


@pytest.mark.parametrize("rows,V", [(1, 1), (5, 2), (3, 31), (40, 33), (300, 1000), (3, 32768), (70, 32768), (9, 32771), (5, 50257),
                                    (2, 131072), (1, 300001), (160, 8192)])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("spread", [0.5, 3.0, 12.0])
def test_sample(lib, rows, V, dt, spread):
    gen = generator(rows * V)
    x = normal(gen, rows, V, dt=dt, scale=spread)
    u = torch.rand(rows, generator=gen, device="cuda")
    for T, k, p, m in ((1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.3, 0, 1.0, 0.05), (0.8, 40, 0.95, 0.02),
                       (2.0, 1000, 0.999, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 1, 0.5, 0.0), (0.0, 5, 0.5, 0.1), (1.0, 0, 1.0, 1.0),
                       (0.05, 0, 0.99999, 0.0), (50.0, 0, 0.5, 0.0), (1.0, V, 0.3, 0.0), (1.0, V - 1, 1.0, 0.0), (3.0, 0, 0.1, 0.5)):
        check_sample(x, u, T, k, p, m)
    no_error()


@pytest.mark.parametrize("dt", [BF, F32])
def test_sample_settings_per_row(lib, dt):
    gen = generator(12)
    rows, V = 200, 4096
    x = normal(gen, rows, V, dt=dt, scale=3.0)
    u, T, p = (torch.rand(rows, generator=gen, device="cuda") for _ in range(3))
    k = torch.randint(-1, 60, (rows,), generator=gen, device="cuda", dtype=I32)
    m = torch.rand(rows, generator=gen, device="cuda") * 0.1
    T[::5], p[::7], m[::3] = 0.0, 1.0, 0.0
    check_sample(x, u, T * 2, k, p, m)
    check_sample(x, u, 1.0, k, p, 0.0)
    check_sample(x, u, T, 10, 0.9, m)
    no_error()


@pytest.mark.parametrize("dt", [BF, F32])
def test_sample_ties(lib, dt):
    """Many equal logits: ranks by index decide, and borders fall inside a run of equal ones."""
    gen = generator(13)
    for V, levels in ((1000, 1), (1000, 3), (5000, 2), (32768, 4), (33, 2), (70000, 1)):
        x = torch.randint(0, levels, (20, V), generator=gen, device="cuda").to(dt)
        u = torch.rand(20, generator=gen, device="cuda")
        u[:4] = torch.tensor([0.0, 0.99999994, 0.5, 0.25], device="cuda")
        for T, k, p, m in ((1.0, 0, 1.0, 0.0), (1.0, 7, 1.0, 0.0), (1.0, 0, 0.5, 0.0), (0.5, V // 2, 0.75, 0.0), (1.0, 0, 1.0, 1.0),
                           (1.0, 100, 0.37, 0.3), (1e-4, 0, 0.9, 0.0), (0.0, 3, 1.0, 0.0)):
            check_sample(x, u, T, k, p, m)


@pytest.mark.parametrize("dt", [BF, F32])
def test_sample_many_close_logits(lib, dt):
    """More logits between two bins' borders than the kernel lists: few distinct values, the largest
    vocabulary, values that differ in their last bits only."""
    gen = generator(18)
    u = torch.rand(3, generator=gen, device="cuda")
    near = (1000 + torch.rand(3, 40000, generator=gen, device="cuda") * 1e-2).to(dt)
    few = (torch.randint(-6, 7, (3, 50000), generator=gen, device="cuda") / 4).to(dt)
    wide = normal(gen, 3, 1 << 19, dt=dt, scale=1.5)
    two = normal(gen, 3, 20000, dt=dt)
    two[:, 1:] = two[:, :-1].clamp(-0.25, 0.25).sign()
    for x in (near, few, wide, two, -near):
        for T, k, p, m in ((1.0, 0, 0.9, 0.0), (0.7, 15000, 1.0, 0.0), (1.3, 19000, 0.6, 0.0), (1e-3, 0, 0.5, 0.0), (30.0, 9999, 0.999, 0.1)):
            check_sample(x, u, T, k, p, m)
    no_error()


@pytest.mark.parametrize("rows,V", [(160, 40000), (2, 1 << 19)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_sample_many_logits_of_a_bin(lib, rows, V, dt):
    """More than 2^14 equal logits of one block, the largest ones or in the middle: the histogram of
    masses overflows there."""
    gen = generator(25 + rows)
    x = normal(gen, rows, V, dt=dt) - 2
    same = torch.rand(rows, V, generator=gen, device="cuda") < torch.linspace(0.3, 0.9, rows, device="cuda")[:, None]
    x[same] = 1.5
    x[::2, 7] = 4.0
    u = torch.rand(rows, generator=gen, device="cuda")
    for T, k, p, m in ((1.0, 0, 0.3, 0.0), (1.0, 0, 0.95, 0.0), (0.8, V // 3, 0.6, 0.0), (2.0, V - 100, 0.999, 0.02)):
        check_sample(x, u, T, k, p, m)
    no_error()


@pytest.mark.parametrize("rows,V", [(1, 32768), (5, 32771), (30, 131072), (60, 32768), (170, 32771), (2, 400001)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_sample_shares_near_one(lib, rows, V, dt):
    """The border of the mass deep in the tail, where the bins about it hold thousands of logits, with
    the lowest drawn tokens among them."""
    gen = generator(19 + rows)
    x = normal(gen, rows, V, dt=dt, scale=2.0)
    u = torch.rand(rows, generator=gen, device="cuda")
    u[::3] = 1 - u[::3] * 1e-4
    u.clamp_(max=0.99999994)
    near = torch.tensor([0.9993, 0.9997, 0.9999, 0.99999, 0.999999, 0.99999994], device="cuda")
    p = near[torch.randint(0, 6, (rows,), generator=gen, device="cuda")]
    for T, k, m in ((1.0, 0, 0.0), (0.8, 0, 1e-3), (2.5, V - V // 8, 0.0), (1.0, V // 2, 1e-4)):
        check_sample(x, u, T, k, p, m)
    check_sample(x, u, 0.8, 0, 0.9999, 0.0)
    no_error()


def test_sample_extremes_of_u(lib):
    x = normal(generator(14), 6, 3001, scale=4.0)
    u = torch.tensor([0.0, 2.0 ** -24, 2.0 ** -30, 0.99999994, 0.5, 1e-38], device="cuda")
    check_sample(x, u)
    check_sample(x, u, 1.0, 3, 0.99, 0.0)


@pytest.mark.parametrize("dt", [BF, F32])
def test_sample_masked_rows(lib, dt):
    """-inf, NaN, +inf, the type's lowest and largest values, signed zeros, rows with nothing left."""
    gen = generator(15)
    x = normal(gen, 10, 500, dt=dt, scale=2.0)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, ::2], x[2, 5] = -math.inf, math.nan
    x[3], x[3, 77] = -math.inf, 1.0
    x[4, 3], x[4, 400], x[4, 7] = math.inf, math.inf, math.nan
    x[5] = torch.finfo(dt).min
    x[6], x[6, 9] = torch.finfo(dt).min, torch.finfo(dt).max
    x[7] = 0.0
    x[7, ::2] = -0.0
    x[8], x[8, 100:] = torch.finfo(dt).tiny, -torch.finfo(dt).tiny
    u = torch.rand(10, generator=gen, device="cuda")
    for T, k, p, m in ((1.0, 0, 1.0, 0.0), (0.7, 3, 0.9, 0.1), (0.0, 0, 1.0, 0.0), (1.0, 250, 0.5, 0.0), (1.0, 0, 0.9, 0.0)):
        check_sample(x, u, T, k, p, m)
    no_error()


def test_sample_bad_settings_are_flagged(lib):
    x = normal(generator(16), 3, 100)
    ok = torch.tensor([0.1, 0.5, 0.9], device="cuda")
    bad = torch.tensor([0.5, math.nan, -1.0], device="cuda")
    token, want = torch.empty(3, dtype=I32, device="cuda"), torch.empty(3, dtype=I32, device="cuda")

    def same(want_how, **how):
        tg.tango_sample(x, how.pop("u", ok), token, **how)
        flagged(8)
        tg.tango_sample(x, want_how.pop("u", ok), want, **want_how)
        no_error()
        assert torch.equal(token, want)
    same(dict(temperature=torch.tensor([0.5, 1.0, 0.0], device="cuda")), temperature=bad)
    same(dict(top_p=torch.tensor([0.5, 1.0, -1.0], device="cuda")), top_p=bad)
    same(dict(min_p=torch.tensor([0.5, 0.0, 1.0], device="cuda")), min_p=torch.tensor([0.5, math.nan, 3.0], device="cuda"))
    same(dict(u=torch.tensor([0.5, 0.0, 0.0], device="cuda")), u=bad)
    same(dict(u=torch.tensor([0.99999994, 0.99999994, 0.2], device="cuda")), u=torch.tensor([1.0, math.inf, 0.2], device="cuda"))


@pytest.mark.parametrize("rows,V", [(3, 37), (200, 500), (2, 32771), (1, 131072)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_sample_extreme_temperatures(lib, dt, rows, V):
    """Temperatures at the ends of their range, down to denormal ones, with equal largest logits and
    masked ones: only the largest are left, or all weigh the same."""
    gen = generator(21 + rows)
    x = normal(gen, rows, V, dt=dt, scale=3.0)
    x[:, ::7] = -math.inf
    x[:, 5], x[:, V // 2 + 1] = 40.0, 40.0
    x[:, 7 * (V // 14)] = 40.0
    u = torch.rand(rows, generator=gen, device="cuda")
    for T in (1e-45, 1e-39, 1.1e-38, 1e-37, 1e30, 3.3e38):
        for k, p, m in ((0, 1.0, 0.0), (5, 1.0, 0.0), (300, 1.0, 0.0), (0, 0.6, 0.0), (V // 2, 0.7, 0.5)):
            check_sample(x, u, T, k, p, m)
            check_sample(x, u, torch.full((rows,), T, device="cuda"), k, p, m)
    no_error()


def test_sample_infinite_temperature_is_flagged(lib):
    """In a row of its own settings it counts as the largest finite one."""
    gen = generator(22)
    x, u = normal(gen, 4, 300), torch.rand(4, generator=gen, device="cuda")
    T = torch.tensor([0.5, math.inf, 1.0, math.inf], device="cuda")
    most = torch.where(T == math.inf, torch.finfo(F32).max, T)
    for how in (dict(), dict(top_k=20), dict(top_p=0.8), dict(top_k=290, top_p=0.5, min_p=0.1)):
        token, want = torch.full((4,), -7, dtype=I32, device="cuda"), torch.full((4,), -8, dtype=I32, device="cuda")
        tg.tango_sample(x, u, token, temperature=T, **how)
        flagged(8)
        tg.tango_sample(x, u, want, temperature=most, **how)
        no_error()
        assert torch.equal(token, want)


def test_sample_top_k_past_32_bits_is_off(lib):
    x, u = normal(generator(23), 50, 200), torch.rand(50, generator=generator(24), device="cuda")
    token, want = torch.empty(50, dtype=I32, device="cuda"), torch.empty(50, dtype=I32, device="cuda")
    tg.tango_sample(x, u, want)
    for k in (2 ** 32 + 1, 2 ** 31, 2 ** 63, -2 ** 32 + 1, -2 ** 40, 200, -1):
        assert torch.equal(tg.tango_sample(x, u, token, top_k=k), want), k


def test_sample_slices(lib):
    """Rows of a padded vocabulary, aligned or not."""
    gen = generator(17)
    for V, pitch, first in ((1000, 1024, 0), (1001, 1003, 1), (32768, 40000, 8)):
        for dt in (BF, F32):
            wide = torch.full((5, pitch), 100.0, dtype=dt, device="cuda")
            wide[:, first:first + V] = normal(gen, 5, V, dt=dt, scale=2.0)
            check_sample(wide[:, first:first + V], torch.rand(5, generator=gen, device="cuda"), 0.9, 0, 0.9, 0.0)


# ---------------------------------------------------------------- together, streams, graphs

def test_training_ends_together(lib):
    """Lookup, norm, tied logits, distillation and back to the tied matrix, against differentiation in
    64 bits."""
    gen = generator(20)
    V, d, N, K, T = 500, 64, 40, 6, 1.5
    E, gamma = normal(gen, V, d, scale=0.3), 1 + normal(gen, d, scale=0.1)
    ids = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=I32)
    ids[5:9] = 17
    ids[-3:] = -1
    t, ti = normal(gen, N, K, scale=2.0), torch.randint(0, V, (N, K), generator=gen, device="cuda", dtype=I32)
    ti[-3:] = -1
    h, x = torch.empty(N, d, device="cuda"), torch.empty(N, d, device="cuda")
    tg.tango_embed(ids, E, h, scale=8.0)
    tg.tango_norm(h, gamma, None, x)
    z = x.double() @ E.double().t()
    z32 = z.float()
    loss, dz = torch.empty(N, device="cuda"), torch.empty_like(z32)
    dloss = torch.full((N,), 1.0 / (N - 3), device="cuda")
    tg.tango_distill_backward(z32, t, ti, dloss, dz, temperature=T, loss=loss)
    dx, dE = (dz.double() @ E.double()).float(), (dz.double().t() @ x.double()).float()
    dh, dgamma = torch.empty_like(dx), torch.empty(d, device="cuda")
    tg.tango_norm_backward(h, gamma, dx, dh, dgamma=dgamma)
    tg.tango_embed_backward(ids, dh, dE, base=dE, scale=8.0)

    E64, g64 = E.double().requires_grad_(), gamma.double().requires_grad_()
    h64 = torch.where((ids >= 0)[:, None], E64[ids.clamp(min=0).long()] * 8.0, 0.0)
    x64 = h64 / (h64.square().mean(-1, keepdim=True) + 1e-6).sqrt() * g64
    l64 = distill_ref(x64 @ E64.t(), t, ti, T)[0]
    (l64 * dloss.double()).sum().backward()
    # every step is fp32 with some tens of roundings
    assert (loss.double() - l64).abs().max() <= 200 * U * l64.abs().max()
    assert (dE.double() - E64.grad).abs().max() <= 500 * U * E64.grad.abs().max()
    assert (dgamma.double() - g64.grad).abs().max() <= 500 * U * g64.grad.abs().max()


def test_example_distills_and_samples(lib):
    """The example's gradients at the model's two ends against differentiation in 64 bits (bf16
    logits, their gradient, x and dx: four roundings of 2^-8, compared in the 2-norm), and its
    sampled tokens."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import generate_tango as ex
    r = ex.distill_step()
    E = r["model"]["embedding"].double().requires_grad_()
    gamma = r["model"]["gamma"].double().requires_grad_()
    h = E[r["ids"].long()]
    x = h / (h.square().mean(-1, keepdim=True) + 1e-6).sqrt() * gamma
    loss = distill_ref(x @ E.t(), r["t_logits"], r["t_ids"], 2.0)[0]
    loss.mean().backward()
    assert ((r["loss"].double() - loss).norm() / loss.norm()).item() <= 4 * 2.0 ** -8
    for got, want in ((r["dE"], E.grad), (r["dgamma"], gamma.grad)):
        assert ((got.double() - want).norm() / want.norm()).item() <= 4 * 2.0 ** -8
    seqs, _ = ex.generate([[1, 2, 3], [7]], 5, temperature=0.9, top_k=20, top_p=0.95)
    again, _ = ex.generate([[1, 2, 3], [7]], 5, temperature=0.9, top_k=20, top_p=0.95)
    assert seqs == again and [len(s) for s in seqs] == [8, 6] and all(0 <= t < ex.VOCAB for s in seqs for t in s)


def _step(b):
    tg.tango_embed(b["ids"], b["E"], b["h"], scale=2.0)
    tg.tango_norm(b["h"], b["gamma"], b["beta"], b["x"], norm=tg.TG_NORM_LAYER)
    tg.tango_distill_backward(b["z"], b["t"], b["ti"], b["dloss"], b["dz"], loss=b["loss"])
    tg.tango_norm_backward(b["h"], b["gamma"], b["x"], b["dh"], norm=tg.TG_NORM_LAYER, dgamma=b["dgamma"], dbeta=b["dbeta"], ws=b["ws1"])
    tg.tango_embed_backward(b["ids"], b["dh"], b["dE"], ws=b["ws2"])
    tg.tango_sample(b["z"], b["u"], b["token"], temperature=0.9, top_k=30, top_p=0.9, logprob=b["logprob"])


def _buffers(seed, N=65, V=3001, d=96, K=7, dt=BF):
    gen = generator(seed)
    z, t, ti = distill_inputs(gen, N, V, K, dt)
    b = dict(ids=torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=I32), E=normal(gen, V, d, dt=dt),
             gamma=normal(gen, d, dt=dt), beta=normal(gen, d, dt=dt), z=z, t=t, ti=ti, u=torch.rand(N, generator=gen, device="cuda"),
             dloss=normal(gen, N))
    out = dict(h=torch.empty(N, d, dtype=dt, device="cuda"), x=torch.empty(N, d, dtype=dt, device="cuda"), dz=torch.empty_like(z),
               loss=torch.empty(N, device="cuda"), dh=torch.empty(N, d, dtype=dt, device="cuda"), dgamma=torch.empty(d, device="cuda"),
               dbeta=torch.empty(d, device="cuda"), dE=torch.empty(V, d, device="cuda"), token=torch.empty(N, dtype=I32, device="cuda"),
               logprob=torch.empty(N, device="cuda"))
    ws = dict(ws1=torch.empty(1 << 22, dtype=torch.uint8, device="cuda"), ws2=torch.empty(1 << 22, dtype=torch.uint8, device="cuda"))
    return b, out, ws


def test_graph_replay_and_other_streams(lib):
    """A captured step, replayed on new inputs, and the same on another stream, give what eager calls
    give, bit for bit."""
    b, out, ws = _buffers(1)
    other, _, _ = _buffers(2)
    _step(b | out | ws)                                     # first use outside of the capture
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        _step(b | out | ws)
    for src in (b, other):
        for n in b:
            b[n].copy_(src[n])
        for t in out.values():
            t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in out.items()}
        _step(b | out | ws)
        torch.cuda.synchronize()
        for n, t in out.items():
            assert torch.equal(got[n], t), n
        for t in out.values():
            t.fill_(3)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            _step(b | out | ws)
        side.synchronize()
        for n, t in out.items():
            assert torch.equal(got[n], t), n
    no_error()


def test_two_streams_at_once(lib):
    """Steps on two streams with their own workspaces do not disturb one another."""
    sets = [_buffers(s, N=200 + s) for s in (3, 4)]
    want = []
    for b, out, ws in sets:
        _step(b | out | ws)
        torch.cuda.synchronize()
        want.append({n: t.clone() for n, t in out.items()})
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        for (b, out, ws), s in zip(sets, streams):
            with torch.cuda.stream(s):
                _step(b | out | ws)
    torch.cuda.synchronize()
    for (b, out, ws), w in zip(sets, want):
        for n, t in out.items():
            assert torch.equal(w[n], t), n


def test_offsets_past_32_bits(lib):
    """Rows that start more than 2^31 elements into their tensor."""
    gen = generator(30)
    V, N = 100_003, 22_000                       # 2.2e9 logits
    z = torch.zeros(N, V, dtype=BF, device="cuda")
    last = normal(gen, 2, V, dt=BF, scale=2.0)
    z[-2:] = last
    u = torch.rand(2, generator=gen, device="cuda")
    token = torch.empty(N, dtype=I32, device="cuda")
    tg.tango_sample(z, torch.cat([torch.rand(N - 2, generator=gen, device="cuda"), u]), token, top_k=40, top_p=0.9)
    assert torch.equal(token[-2:], sample_ref(last, u, 1.0, 40, 0.9, 0.0)[0])
    ids = torch.full((N, 3), -1, dtype=I32, device="cuda")
    ids[-1] = torch.tensor([5, 100_002, 777], device="cuda")
    t, dloss = normal(gen, N, 3), torch.ones(N, device="cuda")
    loss = torch.empty(N, device="cuda")
    tg.tango_distill_backward(z, t, ids, dloss, z, loss=loss)
    check_distill(last[-1:], t[-1:], ids[-1:], 1.0, dloss[-1:], loss[-1:], z[-1:])
    assert (z[:-1] == 0).all() and (loss[:-1] == 0).all()
    del z
    d = 2048
    x = normal(gen, 1_060_000, d, dt=BF)         # 2.17e9 values
    y = torch.empty_like(x)
    tg.tango_norm(x, None, None, y)
    want, n, r = norm_ref(x[-3:], None, None, False, 1e-6)
    within(y[-3:], want, (half_step(BF) * 1.02 + 200 * U) * (want.abs() + 1e-3))
    ids = torch.zeros(len(x), dtype=I32, device="cuda")
    ids[-3:] = 1
    dE = torch.empty(2, d, device="cuda")
    tg.tango_embed_backward(ids, x, dE)
    within(dE[1], x[-3:].double().sum(0), 8 * U * x[-3:].double().abs().sum(0))
    tg.tango_embed(ids, torch.arange(2 * d, device="cuda").view(2, d).to(BF), y)
    assert (y[-1] == torch.arange(d, 2 * d, device="cuda").to(BF)).all() and (y[0] == torch.arange(d, device="cuda").to(BF)).all()


def at_once(calls, times):
    """Makes each of `calls` (returning a status) from a thread of its own, all at the same time; the
    statuses that came back."""
    import threading
    start, seen = threading.Barrier(len(calls)), [set() for _ in calls]

    def work(i):
        start.wait()
        for _ in range(times):
            seen[i].add(calls[i]())
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return set().union(*seen)


def test_norms_of_other_widths_at_once(lib):
    """Host threads that norm rows of different widths, which ask for different amounts of shared memory
    of one kernel, do not disturb one another."""
    import ctypes
    raw, keep, calls = tg.load(), [], []
    for d in (8192, 6148, 7168, 8191, 6147):
        x, y = normal(generator(d), 2, d), torch.empty(2, d, device="cuda")
        p, s = tg.tg_norm_params(2, d, tg.TG_NORM_RMS, 1e-6, 0, tg.TG_F32), torch.cuda.Stream()
        keep.append((x, y, s))
        args = (ctypes.byref(p), x.data_ptr(), None, None, y.data_ptr(), s.cuda_stream)
        calls.append(lambda args=args: raw.tango_norm(*args))
    torch.cuda.synchronize()
    assert at_once(calls, 4000) == {tg.TG_OK}
    for x, y, _ in keep:
        want, n, _ = norm_ref(x, None, None, False, 1e-6)
        within(y, want, (x.shape[1] / 32 + 30) * U * 2 * n.abs())
