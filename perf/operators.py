"""Measured cases of the serving and training operators around the gate aggregation.

Three groups of calls, each in a plain form (elementary torch operations in 32 bits) and
as a user calls the framework:
  rope, rope_bwd  norm of every query and key head with its rotary position, and gradients
  append          this step's keys (normed, rotated) and gates (SiLU) into a paged cache
  paged           TANGO aggregation of the new tokens of ragged sequences over that cache

Sizes: the repository's head geometries (2 heads of 64 with 14,240 or 4,747 gates each, 16
heads of 32 with 1,780 gates each), its batch of 8 x 2,048 tokens and its contexts up to
8,192 tokens; positions, page sizes and ragged mixes are generic.
"""
import math

import numpy as np
import torch

own = False

# ------------------------------------------------------------------------------- cases


def listed():
    return [
        # One decode step of 8 sequences deep into a long context: latency.
        dict(name="rope_step", op="rope", dtype="bf16", rows=8, H=2, Hk=2, d_h=64, rotary=64, layout="half",
             norm="unit", gain=False, far=1000000, factor=16.0, fused=True),
        # Queries and keys of a training batch at the paper's head geometry, as slices of
        # one fused projection.
        dict(name="rope_batch", op="rope", dtype="bf16", rows=65536, H=16, Hk=16, d_h=32, rotary=32, layout="half",
             norm="unit", gain=False, far=8192, factor=1.0, fused=True),
        # Training: gradients with learned norms, interleaved pairs on part of the head.
        dict(name="rope_bwd_batch", op="rope_bwd", dtype="bf16", rows=16384, H=8, Hk=4, d_h=64, rotary=32,
             layout="interleaved", norm="rms", gain=True, far=2048, factor=1.0, fused=False),
        # The fp32 path at an odd number of rows, positions scaled for a long context.
        dict(name="rope_bwd_f32", op="rope_bwd", dtype="f32", rows=5003, H=2, Hk=2, d_h=64, rotary=64, layout="half",
             norm="unit", gain=False, far=131072, factor=8.0, fused=False),
        # One decode step of 32 sequences: one key and 28,480 gates each.
        dict(name="append_step", op="append", dtype="bf16", seqs="1:%s" % ",1:".join(str(65 + 37 * i) for i in range(32)),
             H=2, d_h=64, m_h=14240, pitch=14240, page=16, silu=True, rotary=64, layout="half"),
        # Prefill of a ragged batch in chunks, the three-set gate width at its padded pitch.
        dict(name="append_chunk", op="append", dtype="bf16", seqs="2048:2048,1531:3579,900:900,4000:4096,1:17,713:800",
             H=2, d_h=64, m_h=4747, pitch=4752, page=64, silu=True, rotary=64, layout="half"),
        # One token of one sequence: the smallest call, where latency counts.
        dict(name="paged_step_one", op="paged", dtype="bf16", seqs="1:513", H=2, d_h=64, m_h=14240, pitch=14240,
             page=16, null=False, v=True),
        # One token each of 8 sequences with long caches: the ordinary decode step, bound by memory.
        dict(name="paged_step_batch", op="paged", dtype="bf16",
             seqs="1:8192,1:6001,1:2048,1:4777,1:8191,1:1025,1:7168,1:3300", H=2, d_h=64, m_h=14240, pitch=14240,
             page=64, null=False, v=True),
        # Several tokens each (checked drafts) of 16 sequences at the paper's geometry, with the null gate.
        dict(name="paged_few", op="paged", dtype="bf16",
             seqs=",".join("%d:%d" % (1 + (i * 5) % 8, 150 + 229 * i) for i in range(16)), H=16, d_h=32, m_h=1780,
             pitch=1784, page=16, null=True, v=True),
        # A chunk of a long prompt: 512 new tokens against 8,192 cached ones.
        dict(name="paged_chunk", op="paged", dtype="bf16", seqs="512:8192", H=2, d_h=64, m_h=14240, pitch=14240,
             page=64, null=False, v=True),
        # Fresh prompts, a continued one and decode steps in one batch: bound by the products.
        dict(name="paged_mixed", op="paged", dtype="bf16", seqs="2048:2048,2048:2048,777:1291,1:3001,300:4000,1:64,2048:2048",
             H=2, d_h=64, m_h=14240, pitch=14240, page=32, null=True, v=True),
        # The fp32 path: the three-set gate width, odd lengths, gates alone.
        dict(name="paged_f32", op="paged", dtype="f32", seqs="5:700,1:33,64:64,1:1500", H=2, d_h=64, m_h=4747,
             pitch=4747, page=16, null=True, v=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "paged", "paged", "paged"])
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    if op in ("rope", "rope_bwd"):
        H, d_h = rng.choice([(2, 64), (16, 32), (8, 64), (4, 16), (6, 128)])
        rotary = rng.choice([d_h, d_h // 2, d_h])
        if rng.random() < 0.2:
            rotary = max(2, 2 * rng.randrange(1, d_h // 2 + 1))
        norm = rng.choice(["unit", "unit", "rms"])
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, 32768 if H * d_h <= 256 else 16384), H=H,
                    Hk=rng.choice([H, max(1, H // 2)]), d_h=d_h, rotary=rotary, layout=rng.choice(["half", "interleaved"]),
                    norm=norm, gain=norm == "rms", far=_log(rng, 64, 1000000), factor=rng.choice([1.0, 4.0, 16.0]),
                    fused=rng.random() < 0.5)
    H, d_h, m_h, pitch = rng.choice([(2, 64, 14240, 14240), (16, 32, 1780, 1784), (2, 64, 4747, 4752), (4, 16, 256, 256)])
    if dtype == "f32":
        pitch = m_h if rng.random() < 0.5 else pitch
    page = rng.choice([8, 16, 32, 64, 128])
    m = H * m_h
    if op == "append":
        B, budget, seqs = _log(rng, 1, 32), 60_000_000 // m, []
        for _ in range(B):
            new = min(_log(rng, 1, 2048), max(1, budget // B))
            seqs.append("%d:%d" % (new, new + _log(rng, 1, 128)))
        return dict(op=op, dtype=dtype, seqs=",".join(seqs), H=H, d_h=d_h, m_h=m_h, pitch=pitch, page=page,
                    silu=rng.random() < 0.7, rotary=d_h, layout=rng.choice(["half", "interleaved"]))
    kind = rng.choice(["step", "few", "chunk"])
    seqs, cached, pairs = [], 0, 0
    most = (1.0e9 if dtype == "bf16" else 2.0e8) / m           # cached tokens
    work = (6.0e11 if dtype == "bf16" else 1.0e10) / (2 * m)    # visible pairs
    for _ in range(_log(rng, 1, 24 if kind != "chunk" else 5)):
        new = 1 if kind == "step" else rng.randrange(1, 17) if kind == "few" else _log(rng, 17, 2048)
        length = new + _log(rng, 1, 8192) - 1
        if seqs and (cached + length > most or pairs + new * length > work):
            continue
        length = int(min(length, most))
        new = int(max(1, min(new, length, work // length)))
        cached, pairs = cached + length, pairs + new * length
        seqs.append("%d:%d" % (new, length))
    return dict(op=op, dtype=dtype, seqs=",".join(seqs), H=H, d_h=d_h, m_h=m_h, pitch=pitch, page=page,
                null=rng.random() < 0.4, v=rng.random() < 0.8)


def _seqs(case):
    return [tuple(int(x) for x in s.split(":")) for s in case["seqs"].split(",")]


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# ----------------------------------------------------------------------------- inputs


def _freqs(rotary, factor, dev):
    """Radians per position, 64 bits: base 10,000, positions interpolated by `factor`."""
    c = torch.arange(0, rotary, 2, dtype=torch.float64, device=dev)
    return torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=dev), -c / rotary) / factor


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt, H, d_h = _dt(case), case["H"], case["d_h"]

    def normal(*shape, scale=1.0, dtype=None):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype or dt)

    st = dict(case)
    if case["op"] in ("rope", "rope_bwd"):
        N, Hk = case["rows"], case["Hk"]
        if case["fused"]:
            x = normal(N, (H + Hk) * d_h)
            st["q"], st["k"] = x[:, :H * d_h], x[:, H * d_h:]
        else:
            st["q"], st["k"] = normal(N, H * d_h), normal(N, Hk * d_h)
        st["positions"] = torch.randint(0, case["far"], (N,), generator=gen, device=dev, dtype=torch.int32)
        st["freqs"] = _freqs(case["rotary"], case["factor"], dev)
        st["q_gain"] = 1 + normal(d_h, scale=0.2, dtype=torch.float32) if case["gain"] else None
        st["k_gain"] = 1 + normal(d_h, scale=0.2, dtype=torch.float32) if case["gain"] else None
        if case["op"] == "rope_bwd":
            st["dq_out"], st["dk_out"] = normal(N, H * d_h), normal(N, Hk * d_h)
        return st

    seqs = _seqs(case)
    B, page, m_h, pitch = len(seqs), case["page"], case["m_h"], case["pitch"]
    new = torch.tensor([n for n, _ in seqs])
    lens = torch.tensor([t for _, t in seqs])
    pages = (lens + page - 1) // page
    n_pages, width = int(pages.sum()) + 3, int(pages.max())
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    first = torch.cumsum(pages, 0) - pages
    col = torch.arange(width)
    # unused table entries hold page 0, as a zero-initialised table does
    st["page_table"] = torch.where((col[None] < pages[:, None]).to(dev), order[(first[:, None] + col[None]).clamp(max=n_pages - 1).to(dev)],
                                   torch.zeros((), dtype=torch.int32, device=dev)).contiguous()
    st["lens"] = lens.to(dev, torch.int32)
    st["cu_new"] = torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(new, 0)]).to(dev, torch.int32)
    st["max_new"], st["max_len"], N = int(new.max()), int(lens.max()), int(new.sum())
    st["B"], st["N"] = B, N
    if case["op"] == "append":
        st["k_pages"] = torch.zeros(n_pages, page, H * d_h, dtype=dt, device=dev)
        st["g_pages"] = torch.zeros(n_pages, page, H * pitch, dtype=dt, device=dev)
        st["q"], st["k"] = normal(N, H * d_h), normal(N, H * d_h)
        st["g"] = normal(N, H * pitch)
        st["freqs"] = _freqs(case["rotary"], 1.0, dev)
        return st

    def unit(n):
        x = torch.randn(n, H, d_h, generator=gen, device=dev)
        x = x + 0.5 * torch.randn(H, d_h, generator=gen, device=dev)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt).reshape(n, H * d_h)

    st["k_pages"] = unit(n_pages * page).reshape(n_pages, page, H * d_h)
    g = torch.empty(n_pages, page, H * pitch, dtype=dt, device=dev)
    rows = max(1, (1 << 28) // (page * H * pitch))
    for a in range(0, n_pages, rows):
        g[a:a + rows] = torch.nn.functional.silu(torch.randn(g[a:a + rows].shape, generator=gen, device=dev))
    st["g_pages"] = g
    st["q"] = unit(N)
    st["v"] = normal(N, H * pitch) if case["v"] else None
    st["null_bias"] = normal(H, dtype=torch.float32) if case["null"] else None
    return st


# ------------------------------------------------------------------------- plain forms


def _cos_sin(positions, freqs):
    angle = positions.double()[:, None] * freqs
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def _rotate(z, cos, sin, rotary, layout):
    """z [N, H, d_h] with its first `rotary` columns turned by the rows' angles."""
    z = z.clone()
    a, b = (slice(0, rotary // 2), slice(rotary // 2, rotary)) if layout == "half" else (slice(0, rotary, 2), slice(1, rotary, 2))
    x, y = z[..., a].clone(), z[..., b].clone()
    z[..., a], z[..., b] = x * cos - y * sin, x * sin + y * cos
    return z


def _inv_norm(x, norm):
    if norm == "unit":
        return 1 / x.square().sum(-1, keepdim=True).sqrt().clamp(min=1e-12)
    return 1 / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()


def _norm_rope(x, gain, st, norm, cos, sin):
    x = x.float().reshape(x.shape[0], -1, st["d_h"])
    n = x * _inv_norm(x, norm)
    n = n if gain is None else n * gain
    return _rotate(n, cos, sin, st["rotary"], st["layout"]).flatten(1)


def _norm_rope_bwd(x, dy, gain, st, cos, sin):
    x = x.float().reshape(x.shape[0], -1, st["d_h"])
    r = _inv_norm(x, st["norm"])
    n = x * r
    dz = _rotate(dy.float().reshape(x.shape), cos, -sin, st["rotary"], st["layout"])
    dgain = None if gain is None else (dz.double() * n).sum((0, 1)).float()
    dn = dz if gain is None else dz * gain
    along = (n * dn).sum(-1, keepdim=True) if st["norm"] == "unit" else (n * dn).mean(-1, keepdim=True)
    return (r * (dn - n * along)).flatten(1), dgain


def _token_rows(st):
    """Sequence and position of every new token."""
    row = torch.arange(st["N"], device=st["lens"].device)
    b = torch.searchsorted(st["cu_new"], row.to(torch.int32), right=True).long() - 1
    return b, st["lens"].long()[b] - (st["cu_new"].long()[b + 1] - row)


def _plain_rope(st):
    cos, sin = _cos_sin(st["positions"], st["freqs"])
    dt = _dt(st)
    if st["op"] == "rope":
        return {"q": _norm_rope(st["q"], st["q_gain"], st, st["norm"], cos, sin).to(dt),
                "k": _norm_rope(st["k"], st["k_gain"], st, st["norm"], cos, sin).to(dt)}
    dq, dqg = _norm_rope_bwd(st["q"], st["dq_out"], st["q_gain"], st, cos, sin)
    dk, dkg = _norm_rope_bwd(st["k"], st["dk_out"], st["k_gain"], st, cos, sin)
    out = {"dq": dq.to(dt), "dk": dk.to(dt)}
    return out if dqg is None else out | {"dq_gain": dqg, "dk_gain": dkg}


def _plain_append(st):
    b, pos = _token_rows(st)
    cos, sin = _cos_sin(pos, st["freqs"])
    dt, H, m_h = _dt(st), st["H"], st["m_h"]
    page = st["page_table"].long()[b, pos // st["page"]]
    slot = pos % st["page"]
    g = st["g"].float().reshape(st["N"], H, -1)[..., :m_h]
    g = g / (1 + (-g).exp()) if st["silu"] else g
    gates = st["g_pages"].unflatten(2, (H, -1))[..., :m_h]
    gates[page, slot] = g.to(dt)
    st["k_pages"][page, slot] = _norm_rope(st["k"], None, st, "unit", cos, sin).to(dt)
    return {"q": _norm_rope(st["q"], None, st, "unit", cos, sin).to(dt), "k_pages": st["k_pages"], "g_pages": gates}


def _plain_paged(st):
    """All sequences at once, padded to the longest."""
    B, H, d_h, m_h, page, dev = st["B"], st["H"], st["d_h"], st["m_h"], st["page"], st["lens"].device
    L = st["max_len"]
    b, pos = _token_rows(st)
    r = torch.arange(st["N"], device=dev) - st["cu_new"].long()[b]
    j = torch.arange(L, device=dev)
    table = st["page_table"].long()
    keys = st["k_pages"][table].flatten(1, 2)[:, :L].float().reshape(B, L, H, d_h).transpose(1, 2)
    q = torch.zeros(B, st["max_new"], H, d_h, device=dev)
    q[b, r] = st["q"].float().reshape(-1, H, d_h)
    at = torch.full((B, st["max_new"]), -1, device=dev)
    at[b, r] = pos
    seen = j <= at[..., None]                                              # [B, new, L]
    w = torch.exp(10.0 * (q.transpose(1, 2) @ keys.transpose(2, 3) - 1)) * seen[:, None]  # tau = 10
    den = w.sum(-1, keepdim=True)
    if st["null_bias"] is not None:
        den = den + (st["null_bias"][:, None, None] - 10.0).exp() * (at + 1).float()[:, None, :, None]
    gates = st["g_pages"].unflatten(2, (H, -1))[table].flatten(1, 2)[:, :L, :, :m_h].float()
    gates = torch.where((j < st["lens"][:, None])[..., None, None], gates, gates.new_zeros(())).transpose(1, 2)
    gbar = ((w @ gates) / den).transpose(1, 2)[b, r]                       # [N, H, m_h]
    out = gbar if st["v"] is None else gbar * st["v"].float().reshape(st["N"], H, -1)[..., :m_h]
    return {"out": out.to(_dt(st))}


# ---------------------------------------------------------------------- framework's calls


def _own(st):
    import cross_token_gated_gb300 as tg
    layout = tg.TG_ROPE_HALF if st.get("layout") == "half" else tg.TG_ROPE_INTERLEAVED
    H, m_h = st["H"], st["m_h"] if "m_h" in st else 0
    if st["op"] in ("rope", "rope_bwd"):
        norm = tg.TG_NORM_UNIT if st["norm"] == "unit" else tg.TG_NORM_RMS
        how = dict(H=H, H_k=st["Hk"], positions=st["positions"], layout=layout, norm=norm, q_gain=st["q_gain"],
                   k_gain=st["k_gain"], eps=1e-6)
        dq, dk = (torch.empty(st[n].shape, dtype=st[n].dtype, device=st[n].device) for n in "qk")
        if st["op"] == "rope":
            tg.tango_qk_norm_rope(st["q"], st["k"], dq, dk, st["freqs"], **how)
            return {"q": dq, "k": dk}
        if st["q_gain"] is None:
            tg.tango_qk_norm_rope_backward(st["q"], st["k"], st["dq_out"], st["dk_out"], dq, dk, st["freqs"], **how)
            return {"dq": dq, "dk": dk}
        dqg, dkg = torch.empty_like(st["q_gain"]), torch.empty_like(st["k_gain"])
        tg.tango_qk_norm_rope_backward(st["q"], st["k"], st["dq_out"], st["dk_out"], dq, dk, st["freqs"], dq_gain=dqg,
                                       dk_gain=dkg, **how)
        return {"dq": dq, "dk": dk, "dq_gain": dqg, "dk_gain": dkg}
    if st["op"] == "append":
        q = torch.empty_like(st["q"])
        tg.tango_cache_append(st["q"], st["k"], st["g"], q, st["k_pages"], st["g_pages"], st["page_table"], st["cu_new"],
                              st["lens"], st["freqs"], H=H, m_h=m_h, layout=layout, silu=st["silu"])
        return {"q": q, "k_pages": st["k_pages"], "g_pages": st["g_pages"].unflatten(2, (H, -1))[..., :m_h]}
    out = torch.empty(st["N"], H * st["pitch"], dtype=st["q"].dtype, device=st["q"].device)
    tg.tango_paged_aggregate(st["q"], st["v"], out, st["k_pages"], st["g_pages"], st["page_table"], st["cu_new"], st["lens"],
                             H=H, max_new=st["max_new"], max_len=st["max_len"], s=10.0, null_bias=st["null_bias"], m_h=m_h)
    return {"out": out.unflatten(1, (H, -1))[..., :m_h]}


def run(state):
    if own:
        return _own(state)
    if state["op"] in ("rope", "rope_bwd"):
        return _plain_rope(state)
    return _plain_append(state) if state["op"] == "append" else _plain_paged(state)


# -------------------------------------------------------------------------------- work


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("rope", "rope_bwd"):
        n = case["rows"] * (case["H"] + case["Hk"]) * case["d_h"]
        back = case["op"] == "rope_bwd"
        return {"bytes": n * es * (3 if back else 2) + case["rows"] * 4, "flops": n * (14 if back else 7)}
    seqs = _seqs(case)
    N, m, dqk = sum(n for n, _ in seqs), case["H"] * case["m_h"], case["H"] * case["d_h"]
    if case["op"] == "append":
        return {"bytes": N * (2 * m + 4 * dqk) * es, "flops": N * (m * (4 if case["silu"] else 0) + 14 * dqk)}
    cached = sum(t for _, t in seqs)
    pairs = sum(n * t - n * (n - 1) // 2 for n, t in seqs)
    return {"bytes": (cached * (m + dqk) + N * (dqk + m * (2 if case["v"] else 1))) * es,
            "flops": 2 * pairs * (m + dqk) + N * m * 2}


# ------------------------------------------------------------- definitions in 64 bits


def _turned(z, positions, freqs, rotary, layout, sign):
    """Rotation as a complex product."""
    e = torch.polar(torch.ones_like(freqs).expand(len(positions), -1), sign * positions.double()[:, None] * freqs)
    head = z[..., :rotary]
    if layout == "half":
        c = torch.complex(head[..., :rotary // 2].contiguous(), head[..., rotary // 2:].contiguous()) * e[:, None]
        head = torch.cat([c.real, c.imag], -1)
    else:
        c = torch.view_as_complex(head.reshape(*z.shape[:-1], rotary // 2, 2).contiguous()) * e[:, None]
        head = torch.view_as_real(c).reshape(*z.shape[:-1], rotary)
    return torch.cat([head, z[..., rotary:]], -1)


def _length(x, norm):
    if norm == "unit":
        return torch.linalg.vector_norm(x, dim=-1, keepdim=True).clamp(min=1e-12)
    return torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6)


def _exact_rope(st, x, gain, norm, positions):
    x = x.double().unflatten(1, (-1, st["d_h"]))
    z = x / _length(x, norm) * (1.0 if gain is None else gain.double())
    return _turned(z, positions, st["freqs"], st["rotary"], st["layout"], 1.0).flatten(1)


def _exact_rope_bwd(st, x, dy, gain):
    """The Jacobian of x / |x| (or of x / rms) applied to the gradient turned back."""
    x = x.double().unflatten(1, (-1, st["d_h"]))
    dz = _turned(dy.double().unflatten(1, (-1, st["d_h"])), st["positions"], st["freqs"], st["rotary"], st["layout"], -1.0)
    s = _length(x, st["norm"])
    dgain = None if gain is None else torch.einsum("nhc,nhc->c", dz, x / s)
    dn = dz * (1.0 if gain is None else gain.double())
    share = 1.0 if st["norm"] == "unit" else 1.0 / x.shape[-1]
    dx = dn / s - x * ((x * dn).sum(-1, keepdim=True) * share / s ** 3)
    return dx.flatten(1), dgain


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return {n: _exact_rope(st, st[n], st[n + "_gain"], st["norm"], st["positions"]) for n in "qk"}
    if case["op"] == "rope_bwd":
        dq, dqg = _exact_rope_bwd(st, st["q"], st["dq_out"], st["q_gain"])
        dk, dkg = _exact_rope_bwd(st, st["k"], st["dk_out"], st["k_gain"])
        return {"dq": dq, "dk": dk} if dqg is None else {"dq": dq, "dk": dk, "dq_gain": dqg, "dk_gain": dkg}
    H, m_h, d_h, page = case["H"], case["m_h"], case["d_h"], case["page"]
    seqs, dev = _seqs(case), st["lens"].device
    starts = np.concatenate([[0], np.cumsum([n for n, _ in seqs])])
    where = [st["page_table"][b, torch.arange(t, device=dev) // page].long() * page + torch.arange(t, device=dev) % page
             for b, (_, t) in enumerate(seqs)]
    if case["op"] == "append":
        pos = torch.cat([torch.arange(t - n, t, device=dev) for n, t in seqs])
        slots = torch.cat([w[t - n:] for w, (n, t) in zip(where, seqs)])
        k = st["k_pages"].double()
        k.view(-1, H * d_h)[slots] = _exact_rope(st, st["k"], None, "unit", pos)
        g = torch.zeros(*st["g_pages"].shape[:2], H, m_h, dtype=torch.float64, device=dev)
        x = st["g"].unflatten(1, (H, -1))[..., :m_h].double()
        g.view(-1, H, m_h)[slots] = x * torch.sigmoid(x) if case["silu"] else x
        return {"q": _exact_rope(st, st["q"], None, "unit", pos), "k_pages": k, "g_pages": g}
    out = torch.empty(st["N"], H, m_h, dtype=torch.float64, device=dev)
    keys, gates = st["k_pages"].view(-1, H, d_h), st["g_pages"].unflatten(2, (H, -1)).flatten(0, 1)
    for b, (n, t) in enumerate(seqs):
        rows = slice(int(starts[b]), int(starts[b + 1]))
        at = torch.arange(t - n, t, device=dev)
        for a in range(H):
            logit = 10.0 * st["q"][rows].double().view(n, H, d_h)[:, a] @ keys[where[b], a].double().T
            logit = logit.masked_fill(torch.arange(t, device=dev) > at[:, None], -math.inf)
            total = torch.logsumexp(logit, 1)
            if st["null_bias"] is not None:
                total = torch.logaddexp(total, st["null_bias"][a].double() + (at + 1).double().log())
            out[rows, a] = torch.exp(logit - total[:, None]) @ gates[where[b], a, :m_h].double()
    return {"out": out if st["v"] is None else out * st["v"].double().unflatten(1, (H, -1))[..., :m_h]}
