"""Measured cases of the operators at the two ends of the language model.

Four groups of calls, each in a plain form (elementary torch operations in 32 bits, 64 where
they decide about whole numbers or sum over all rows) and as a user calls the framework:
  embed, embed_bwd       token lookup with scaling, and the embedding's gradient
  norm, norm_bwd         RMS and layer norm, gradients of the input, the gain and the bias
  distill, distill_grad, distill_both
                         distillation from a teacher's top logits: loss, loss and gradient from
                         one call, loss and then gradient from saved statistics
  sample                 temperature, top-k, top-p and min-p from given uniform numbers

Sizes: the repository's batch of 8 x 2,048 tokens, its widths 512 and 768 and its vocabulary
of 32,768; the number of a teacher's logits, of sampled rows and other vocabularies are generic.
"""
import math

import numpy as np
import torch

own = False
FLOOR = 2.0 ** -40  # a token with less than this share of the largest weight is never drawn

# ------------------------------------------------------------------------------- cases


def listed():
    return [
        # Token lookup of one decode step of 32 sequences: latency.
        dict(name="embed_step", op="embed", dtype="bf16", rows=32, d=512, vocab=32768, scale=22.627417, pads=0.0),
        # The embedding's gradient of a training batch of 8 x 2,048 tokens, frequent tokens among them.
        dict(name="embed_bwd_batch", op="embed_bwd", dtype="bf16", grad="f32", rows=16384, d=512, vocab=32768, scale=1.0,
             pads=0.0, accumulate=False),
        # The fp32 path added to the tied matrix's gradient, an odd number of tokens, padded sequences.
        dict(name="embed_bwd_f32", op="embed_bwd", dtype="f32", grad="f32", rows=5003, d=768, vocab=32768, scale=27.712813,
             pads=0.15, accumulate=True),
        # Layer norm of a large batch of tokens.
        dict(name="norm_batch", op="norm", dtype="bf16", rows=65536, d=768, norm="layer", bias=True, slice=False),
        # Training: the model's RMSNorm, its input's gradient joined with the residual's, its gain's gradient.
        dict(name="norm_bwd_batch", op="norm_bwd", dtype="bf16", rows=16384, d=512, norm="rms", bias=False, residual=True,
             slice=False),
        # The fp32 path of the layer norm at an odd number of rows.
        dict(name="norm_bwd_f32", op="norm_bwd", dtype="f32", rows=5003, d=768, norm="layer", bias=True, residual=False,
             slice=False),
        # The loss of a validation batch.
        dict(name="distill_loss", op="distill", dtype="bf16", rows=8192, vocab=32768, k=64, temperature=2.0, pads=0.05),
        # Training: loss and gradient of 8 x 2,048 tokens from one call.
        dict(name="distill_batch", op="distill_grad", dtype="bf16", rows=16384, vocab=32768, k=64, temperature=1.0, pads=0.05),
        # The fp32 path, loss first and gradient afterwards, at a vocabulary whose rows are not aligned.
        dict(name="distill_f32", op="distill_both", dtype="f32", rows=1003, vocab=32771, k=17, temperature=1.5, pads=0.0),
        # One sequence's next token: the smallest call, where latency counts.
        dict(name="sample_one", op="sample", dtype="bf16", rows=1, vocab=32768, spread=2.5, temperature=0.8, top_k=0,
             top_p=0.95, min_p=0.0, mixed=False, banned=0),
        # A serving batch whose requests each bring their own settings.
        dict(name="sample_batch", op="sample", dtype="bf16", rows=256, vocab=32768, spread=2.5, temperature=0.8, top_k=50,
             top_p=0.9, min_p=0.02, mixed=True, banned=40),
        # fp32 logits, nearly flat, drawn from a large nucleus: most tokens stay candidates.
        dict(name="sample_f32", op="sample", dtype="f32", rows=61, vocab=32771, spread=1.0, temperature=1.2, top_k=0,
             top_p=0.98, min_p=0.0, mixed=False, banned=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _vocab(rng):
    return rng.choice([32768, 32768, 32771, 50257, 1000, _log(rng, 1000, 131072)])


def draw(rng):
    group = rng.choice(["embed", "norm", "distill", "sample"])
    dtype = "bf16" if rng.random() < 0.7 else "f32"
    if group == "embed":
        d = rng.choice([512, 768, 512, 256, 1000, _log(rng, 32, 2048)])
        vocab = rng.choice([32768, 1000, 50257, _log(rng, 256, 65536)])
        rows = min(_log(rng, 1, 65536), 33_000_000 // d)
        case = dict(op=rng.choice(["embed", "embed_bwd", "embed_bwd"]), dtype=dtype, rows=rows, d=d, vocab=vocab,
                    scale=rng.choice([1.0, math.sqrt(d)]), pads=rng.choice([0.0, 0.0, 0.2]))
        if case["op"] == "embed_bwd":
            case["grad"], case["accumulate"] = rng.choice(["f32", "f32", dtype]), rng.random() < 0.4
        return case
    if group == "norm":
        d = rng.choice([512, 768, 1024, 4096, 100, 2049, _log(rng, 16, 8192)])
        layer, back = rng.random() < 0.5, rng.random() < 0.6
        case = dict(op="norm_bwd" if back else "norm", dtype=dtype, rows=min(_log(rng, 1, 65536), 50_000_000 // d), d=d,
                    norm="layer" if layer else "rms", bias=layer and rng.random() < 0.8, slice=rng.random() < 0.3)
        if back:
            case["residual"] = rng.random() < 0.5
        return case
    if group == "distill":
        vocab = _vocab(rng)
        rows = min(_log(rng, 1, 16384), (500_000_000 if dtype == "bf16" else 250_000_000) // vocab)
        return dict(op=rng.choice(["distill", "distill_grad", "distill_grad", "distill_both"]), dtype=dtype, rows=rows,
                    vocab=vocab, k=_log(rng, 1, 256), temperature=rng.choice([1.0, 2.0, 1.5, 0.7]),
                    pads=rng.choice([0.0, 0.1]))
    return dict(op="sample", dtype=dtype, rows=_log(rng, 1, 256), vocab=_vocab(rng), spread=rng.choice([1.0, 2.5, 5.0]),
                temperature=rng.choice([1.0, 0.7, 1.3, 0.0]), top_k=rng.choice([0, 0, 1, 20, 50, 1000]),
                top_p=rng.choice([1.0, 0.95, 0.8, 0.99]), min_p=rng.choice([0.0, 0.0, 0.05]), mixed=rng.random() < 0.4,
                banned=rng.choice([0, 0, 100]))


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


# ----------------------------------------------------------------------------- inputs


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt, op = _dt(case["dtype"]), case["op"]

    def normal(*shape, scale=1.0, dtype=None):
        out = torch.empty(*shape, dtype=dtype or dt, device=dev)
        flat, step = out.view(-1), 1 << 27
        for a in range(0, flat.numel(), step):
            flat[a:a + step] = torch.randn(min(step, flat.numel() - a), generator=gen, device=dev) * scale
        return out

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    st = dict(case)
    if op in ("embed", "embed_bwd"):
        N, d, V = case["rows"], case["d"], case["vocab"]
        # frequencies as 1 / rank, ranks spread over the ids
        rank = (torch.exp(uniform(N) * math.log(V)) - 1).long().clamp(0, V - 1)
        ids = (torch.randperm(V, generator=gen, device=dev)[rank]).to(torch.int32)
        st["ids"] = torch.where(uniform(N) < case["pads"], torch.full_like(ids, -1), ids)
        if op == "embed":
            st["E"] = normal(V, d, scale=0.02)
        else:
            st["dout"] = normal(N, d)
            st["dE"] = normal(V, d, scale=0.1, dtype=_dt(case["grad"])) if case["accumulate"] else None
        return st
    if op in ("norm", "norm_bwd"):
        N, d = case["rows"], case["d"]
        if case["slice"]:
            st["x"] = normal(N, 2 * d, scale=1.5)[:, :d]
        else:
            st["x"] = normal(N, d, scale=1.5)
        st["gamma"] = (1 + 0.2 * torch.randn(d, generator=gen, device=dev)).to(dt)
        st["beta"] = normal(d, scale=0.1) if case["bias"] else None
        if op == "norm_bwd":
            st["dy"] = normal(N, d)
            st["dres"] = normal(N, d) if case["residual"] else None
        return st
    if op.startswith("distill"):
        N, V, K = case["rows"], case["vocab"], case["k"]
        st["logits"] = normal(N, V, scale=2.5)
        t, ids = torch.empty(N, K, device=dev), torch.empty(N, K, dtype=torch.int32, device=dev)
        step = max(1, (1 << 26) // V)
        for a in range(0, N, step):
            part = st["logits"][a:a + step].float()
            part = part + torch.randn(part.shape, generator=gen, device=dev)
            v, i = part.topk(K, dim=1)
            t[a:a + step], ids[a:a + step] = v, i.to(torch.int32)
        st["t_logits"] = t
        st["t_ids"] = torch.where((uniform(N) < case["pads"])[:, None], torch.full_like(ids, -1), ids)
        if op != "distill":
            st["dloss"] = uniform(N) * (2.0 / N)
        return st
    N, V = case["rows"], case["vocab"]
    x = normal(N, V, scale=case["spread"])
    if case["banned"]:
        x.view(-1)[torch.randint(0, N * V, (case["banned"] * N,), generator=gen, device=dev)] = -math.inf
    st["logits"], st["uniform"] = x, uniform(N)
    if case["mixed"]:  # each request its own settings, some of them off
        off = uniform(4, N) < 0.3
        st["temperature"] = torch.where(off[0], torch.zeros(N, device=dev), case["temperature"] * (0.5 + uniform(N)))
        st["top_k"] = torch.where(off[1], 0, torch.randint(1, max(2, 2 * case["top_k"]), (N,), generator=gen, device=dev)).to(torch.int32)
        st["top_p"] = torch.where(off[2], torch.ones(N, device=dev), case["top_p"] + (1 - case["top_p"]) * uniform(N))
        st["min_p"] = torch.where(off[3], torch.zeros(N, device=dev), 2 * case["min_p"] * uniform(N))
    return st


# ------------------------------------------------------------------------- plain forms


def _plain_embed(st):
    ids, dt = st["ids"].long(), _dt(st["dtype"])
    keep = ids != -1
    if st["op"] == "embed":
        rows = st["E"][ids.clamp(min=0)].float() * st["scale"]
        return {"out": torch.where(keep[:, None], rows, rows.new_zeros(())).to(dt)}
    g = torch.zeros(st["vocab"], st["d"], device=ids.device)
    g.index_add_(0, ids[keep], st["dout"].float()[keep])
    g = g * st["scale"]
    if st["dE"] is not None:
        g = g + st["dE"].float()
    return {"dE": g.to(_dt(st["grad"]))}


def _plain_norm(st):
    x, dt, layer = st["x"].float(), _dt(st["dtype"]), st["norm"] == "layer"
    g = st["gamma"].float()
    c = x - x.mean(-1, keepdim=True) if layer else x
    r = 1 / (c.square().mean(-1, keepdim=True) + 1e-5).sqrt()
    n = c * r
    if st["op"] == "norm":
        y = n * g
        return {"y": (y if st["beta"] is None else y + st["beta"].float()).to(dt)}
    dy = st["dy"].float()
    dn = dy * g
    dx = dn - n * (dn * n).mean(-1, keepdim=True)
    if layer:
        dx = dx - dn.mean(-1, keepdim=True)
    dx = dx * r
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    out = {"dx": dx.to(dt), "dgamma": (dy.double() * n).sum(0).float()}
    return out if st["beta"] is None else out | {"dbeta": dy.double().sum(0).float()}


def _plain_distill(st):
    T, ids = st["temperature"], st["t_ids"].long()
    live = ids >= 0
    t = torch.where(live, st["t_logits"], torch.full_like(st["t_logits"], -math.inf))
    any_live = live.any(-1, keepdim=True)
    e = torch.where(live, ((t - torch.where(any_live, t.amax(-1, keepdim=True), 0.0)) / T).exp(), 0.0)
    p = e / torch.where(any_live, e.sum(-1, keepdim=True), 1.0)
    logp = torch.where(p > 0, p, 1.0).log()
    z = st["logits"].float()
    z = (z - z.amax(-1, keepdim=True)) / T
    w = z.exp()
    total = w.sum(-1, keepdim=True)
    logq = z.gather(1, ids.clamp(min=0)) - total.log()
    loss = T * T * torch.where(p > 0, p * (logp - logq), 0.0).sum(-1)
    if st["op"] == "distill":
        return {"loss": loss}
    d = w * torch.where(any_live, 1 / total, 0.0)
    d.scatter_add_(1, ids.clamp(min=0), -p)
    return {"loss": loss, "dlogits": (d * (st["dloss"] * T)[:, None]).to(st["logits"].dtype)}


def _settings(st, dev):
    """Every row's temperature, top-k, top-p and min-p."""
    N = st["rows"]
    return [st[n] if torch.is_tensor(st[n]) else torch.full((N,), float(st[n]), device=dev)
            for n in ("temperature", "top_k", "top_p", "min_p")]


def _plain_sample(st):
    """In 64 bits: a token is a whole number, and weights next to a border decide it."""
    x, V = st["logits"].float(), st["vocab"]
    T, k, p, m = (s.double()[:, None] for s in _settings(st, x.device))
    top = x.amax(-1, keepdim=True)
    w = ((x.double() - top) / torch.where(T > 0, T, 1.0)).exp()
    w = torch.where(T > 0, w, (torch.arange(V, device=x.device) == x.argmax(-1, keepdim=True)).double())
    w = torch.where(w >= FLOOR, w, 0.0)
    order = x.sort(dim=-1, descending=True, stable=True).indices
    s = w.gather(1, order)
    rank = torch.arange(V, device=x.device)
    s = torch.where((k <= 0) | (rank < k), s, 0.0)
    before = s.cumsum(-1) - s
    total = s.sum(-1, keepdim=True)
    s = torch.where((p >= 1) | (before < p * total) | (rank == 0), s, 0.0)
    s = torch.where((s >= m) | (rank == 0), s, 0.0)
    w = torch.zeros_like(w).scatter_(1, order, s)
    c = w.cumsum(-1)
    total = c[:, -1:]
    token = (c <= st["uniform"].double()[:, None] * total).sum(-1).clamp(max=V - 1)
    drawn = w.gather(1, token[:, None])
    return {"token": token.to(torch.int32), "logprob": (drawn / total).log()[:, 0].float()}


# ---------------------------------------------------------------------- framework's calls


def _own(st):
    import cross_token_gated_gb300 as tg
    op = st["op"]
    if op == "embed":
        out = torch.empty(st["rows"], st["d"], dtype=st["E"].dtype, device=st["E"].device)
        return {"out": tg.tango_embed(st["ids"], st["E"], out, scale=st["scale"], pad_id=-1)}
    if op == "embed_bwd":
        dE = torch.empty(st["vocab"], st["d"], dtype=_dt(st["grad"]), device=st["dout"].device)
        tg.tango_embed_backward(st["ids"], st["dout"], dE, scale=st["scale"], pad_id=-1, base=st["dE"])
        return {"dE": dE}
    if op in ("norm", "norm_bwd"):
        how = dict(norm=tg.TG_NORM_LAYER if st["norm"] == "layer" else tg.TG_NORM_RMS, eps=1e-5)
        out = torch.empty(st["rows"], st["d"], dtype=st["x"].dtype, device=st["x"].device)
        if op == "norm":
            return {"y": tg.tango_norm(st["x"], st["gamma"], st["beta"], out, **how)}
        dgamma = torch.empty(st["d"], device=out.device)
        dbeta = None if st["beta"] is None else torch.empty_like(dgamma)
        tg.tango_norm_backward(st["x"], st["gamma"], st["dy"], out, dres=st["dres"], dgamma=dgamma, dbeta=dbeta, **how)
        return {"dx": out, "dgamma": dgamma} | ({} if dbeta is None else {"dbeta": dbeta})
    if op.startswith("distill"):
        z, how = st["logits"], dict(temperature=st["temperature"])
        teacher, loss = (st["t_logits"], st["t_ids"]), torch.empty(st["rows"], device=z.device)
        if op == "distill":
            return {"loss": tg.tango_distill(z, *teacher, loss, **how)}
        dz = torch.empty_like(z)
        if op == "distill_grad":
            tg.tango_distill_backward(z, *teacher, st["dloss"], dz, loss=loss, **how)
        else:
            stats = torch.empty(st["rows"], 2, device=z.device)
            tg.tango_distill(z, *teacher, loss, stats=stats, **how)
            tg.tango_distill_backward(z, *teacher, st["dloss"], dz, stats=stats, **how)
        return {"loss": loss, "dlogits": dz}
    token = torch.empty(st["rows"], dtype=torch.int32, device=st["logits"].device)
    logprob = torch.empty(st["rows"], device=token.device)
    tg.tango_sample(st["logits"], st["uniform"], token, temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                    min_p=st["min_p"], logprob=logprob)
    return {"token": token, "logprob": logprob}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op in ("embed", "embed_bwd"):
        return _plain_embed(state)
    if op in ("norm", "norm_bwd"):
        return _plain_norm(state)
    return _plain_sample(state) if op == "sample" else _plain_distill(state)


# -------------------------------------------------------------------------------- work


def work(case):
    es, op, N = 2 if case["dtype"] == "bf16" else 4, case["op"], case["rows"]
    if op == "embed":
        return {"bytes": N * (case["d"] * 2 * es + 4), "flops": N * case["d"]}
    if op == "embed_bwd":
        gs = (2 if case["grad"] == "bf16" else 4) * (2 if case["accumulate"] else 1)
        return {"bytes": N * (case["d"] * es + 4) + case["vocab"] * case["d"] * gs, "flops": (N + case["vocab"]) * case["d"]}
    if op in ("norm", "norm_bwd"):
        back = op == "norm_bwd"
        return {"bytes": N * case["d"] * es * (2 + (1 + case["residual"] if back else 0)), "flops": N * case["d"] * (13 if back else 7)}
    if op.startswith("distill"):
        n = N * case["vocab"]
        return {"bytes": n * es * (1 if op == "distill" else 2) + N * case["k"] * 8, "flops": n * (4 if op == "distill" else 6)}
    return {"bytes": N * (case["vocab"] * es + 12), "flops": N * case["vocab"] * 6}


# ------------------------------------------------------------- definitions in 64 bits


def _exact_embed(st):
    ids = st["ids"].long()
    if st["op"] == "embed":
        out = torch.zeros(st["rows"], st["d"], dtype=torch.float64, device=ids.device)
        at = (ids >= 0).nonzero()[:, 0]
        out[at] = st["E"].double()[ids[at]] * st["scale"]
        return {"out": out}
    # running sums of the rows in the order of their tokens, read at each token's end
    order = torch.argsort(ids, stable=True)
    sums = torch.cat([torch.zeros(1, st["d"], dtype=torch.float64, device=ids.device),
                      st["dout"].double()[order].cumsum(0)])
    ends = torch.searchsorted(ids[order], torch.arange(-1, st["vocab"], device=ids.device), right=True)
    g = (sums[ends[1:]] - sums[ends[:-1]]) * st["scale"]
    return {"dE": g if st["dE"] is None else g + st["dE"].double()}


def _exact_norm(st):
    x, g, d = st["x"].double(), st["gamma"].double(), st["d"]
    mu = x.sum(-1, keepdim=True) / d if st["norm"] == "layer" else 0.0
    s = torch.sqrt(((x - mu) ** 2).sum(-1, keepdim=True) / d + 1e-5)
    if st["op"] == "norm":
        return {"y": (x - mu) / s * g + (0.0 if st["beta"] is None else st["beta"].double())}
    # the Jacobian of (x - mu) / s applied to the gradient
    dy = st["dy"].double()
    dn = dy * g
    dx = dn / s - (x - mu) * (((x - mu) * dn).sum(-1, keepdim=True) / (d * s ** 3))
    if st["norm"] == "layer":
        dx = dx - (dn / s).sum(-1, keepdim=True) / d
    out = {"dx": dx if st["dres"] is None else dx + st["dres"].double(), "dgamma": torch.einsum("nc,nc->c", dy, (x - mu) / s)}
    return out if st["beta"] is None else out | {"dbeta": torch.einsum("nc->c", dy)}


def _exact_distill(st):
    N, V, T = st["rows"], st["vocab"], float(st["temperature"])
    dev, grad = st["logits"].device, st["op"] != "distill"
    loss = torch.zeros(N, dtype=torch.float64, device=dev)
    dz = torch.zeros(N, V, dtype=torch.float64, device=dev) if grad else None
    rows = (st["t_ids"][:, 0] >= 0).nonzero()[:, 0]
    for part in rows.split(max(1, (1 << 26) // V)):
        ids = st["t_ids"][part].long()
        logp = torch.log_softmax(st["t_logits"][part].double() / T, -1)
        logq = torch.log_softmax(st["logits"][part].double() / T, -1)
        loss[part] = T * T * (logp.exp() * (logp - logq.gather(1, ids))).sum(-1)
        if grad:
            target = torch.zeros_like(logq).scatter_add_(1, ids, logp.exp())
            dz[part] = (logq.exp() - target) * (T * st["dloss"][part].double()[:, None])
    return {"loss": loss, "dlogits": dz} if grad else {"loss": loss}


def _exact_sample(st):
    """Row by row on the host."""
    x = st["logits"].double().cpu().numpy()
    T, k, p, m = (s.double().cpu().numpy() for s in _settings(st, st["logits"].device))
    u = st["uniform"].double().cpu().numpy()
    token, logprob = np.zeros(len(x), np.int32), np.zeros(len(x))
    for i, row in enumerate(x):
        if T[i] == 0:
            token[i] = int(np.argmax(row))
            continue
        kept = np.argsort(-row, kind="stable")
        kept = kept[np.exp((row[kept] - row[kept[0]]) / T[i]) >= FLOOR]
        if k[i] > 0:
            kept = kept[:int(k[i])]
        w = np.exp((row[kept] - row[kept[0]]) / T[i])
        n = len(kept)
        if p[i] < 1:
            n = 1 + int(np.searchsorted(np.cumsum(w), p[i] * math.fsum(w)))
        n = max(1, min(n, len(kept), int((w >= m[i]).sum())))
        kept = np.sort(kept[:n])
        w = np.exp((row[kept] - row.max()) / T[i])
        total = math.fsum(w)
        j = min(n - 1, int(np.searchsorted(np.cumsum(w), u[i] * total, side="right")))
        token[i], logprob[i] = kept[j], math.log(w[j] / total)
    dev = st["logits"].device
    return {"token": torch.from_numpy(token).to(dev), "logprob": torch.from_numpy(logprob).to(dev)}


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op in ("embed", "embed_bwd"):
        return _exact_embed(st)
    if op in ("norm", "norm_bwd"):
        return _exact_norm(st)
    return _exact_sample(st) if op == "sample" else _exact_distill(st)
