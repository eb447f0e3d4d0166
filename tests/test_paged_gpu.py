"""The paged cache: append and aggregation of ragged batches against float64.

Tolerances of an aggregated value out = v * N / D, N = sum w g, D = sum w (+ null): the
stored value is off by half a step of its type (bf16 2^-8, fp32 2^-24).  The weights are
fp32 (relative error at most tau (d_h + 4) 2^-23 from the d_h-term dot product, the
exponent's argument and exp2) and, on the tensor cores, rounded to bf16 (2^-8 each); D sums
the weights as applied, so N / D is off by at most twice a weight's relative error times
A = sum w |g| / D.  Sums in fp32 add n 2^-24 A for n terms in the worst case; the terms here
are added in at most 2^11 groups, so 2^-13 A bounds them for every length tested.
"""
import math

import pytest
import torch

import cross_token_gated_gb300 as tg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SUMS = {"bf16": 2.0 ** -13, "f32": 2.0 ** -20}


class Batch:
    """A ragged batch over a pool whose unused slots hold NaN, pages in shuffled order."""

    def __init__(self, seqs, H, d_h, m_h, dtype, page, pitch=None, seed=0, tau=10.0, fill=True, extra=3):
        g = torch.Generator().manual_seed(seed)
        dt = DT[dtype]
        self.seqs, self.H, self.d_h, self.m_h, self.dtype, self.page = seqs, H, d_h, m_h, dtype, page
        self.pitch = pitch or m_h
        self.B, self.N = len(seqs), sum(n for n, _ in seqs)
        need = [max(0, -(-t // page)) for _, t in seqs]
        width = max(max(need), 1) + 1
        pool = sum(need) + extra
        order = torch.randperm(pool, generator=g).tolist()
        # entries past a sequence's pages are not page numbers at all
        table = torch.full((self.B, width), -7, dtype=torch.int32)
        self.k_pages = torch.full((pool, page, H * d_h), math.nan, dtype=dt)
        self.g_pages = torch.full((pool, page, H * self.pitch), math.nan, dtype=dt)
        self.keys, self.gates = [], []
        for b, (n, t) in enumerate(seqs):
            pages = [order.pop() for _ in range(need[b])]
            table[b, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
            t = max(t, 0)
            k = torch.randn(t, H, d_h, generator=g)
            k = (k / k.norm(dim=-1, keepdim=True).clamp(min=1e-6)).to(dt)
            x = torch.randn(t, H, m_h, generator=g).to(dt)
            self.keys.append(k)
            self.gates.append(x)
            if fill:
                for j in range(t):
                    self.k_pages[pages[j // page], j % page] = k[j].flatten()
                    self.g_pages[pages[j // page], j % page].view(H, self.pitch)[:, :m_h] = x[j]
        q = torch.randn(self.N, H, d_h, generator=g)
        self.q = (q / q.norm(dim=-1, keepdim=True)).to(dt).reshape(self.N, -1).cuda()
        self.v = torch.randn(self.N, H * self.pitch, generator=g).to(dt).cuda()
        self.table, self.k_pages, self.g_pages = table.cuda(), self.k_pages.cuda(), self.g_pages.cuda()
        self.cu = torch.tensor([0] + [n for n, _ in seqs]).cumsum(0).to(torch.int32).cuda()
        self.lens = torch.tensor([t for _, t in seqs], dtype=torch.int32).cuda()
        self.max_new, self.max_len = max(1, max(n for n, _ in seqs)), max(1, max(t for _, t in seqs))

    def run(self, v=True, tau=None, s=10.0, null=None, **kw):
        out = torch.full((self.N, self.H * self.pitch), 5.0, dtype=DT[self.dtype], device="cuda")
        args = dict(H=self.H, max_new=self.max_new, max_len=self.max_len, s=s, tau=tau, null_bias=null, m_h=self.m_h)
        args.update(kw)
        tg.tango_paged_aggregate(self.q, (self.v if v is True else v) if v is not False else None, out, self.k_pages,
                                 self.g_pages, self.table, self.cu, self.lens, **args)
        return out

    def want(self, v=True, tau=None, s=10.0, null=None):
        """(out, tolerance scale A |v|) in float64, [N, H, m_h]; rows without keys are 0."""
        H, out, mag = self.H, [], []
        taus = [s] * H if tau is None else tau.tolist()
        row = 0
        for b, (n, t) in enumerate(self.seqs):
            k, g = self.keys[b].double(), self.gates[b].double()
            q = self.q[row:row + n].double().cpu().view(n, H, self.d_h)
            pos = torch.arange(t - n, t)
            seen = torch.arange(max(t, 0))[None] <= pos[:, None]
            o, a = torch.zeros(n, H, self.m_h, dtype=torch.float64), torch.zeros(n, H, self.m_h, dtype=torch.float64)
            for h in range(H):
                w = torch.where(seen, (taus[h] * (q[:, h] @ k[:, h].T - 1)).exp(), torch.zeros((), dtype=torch.float64))
                den = w.sum(1)
                if null is not None:
                    den = den + (pos + 1).clamp(min=0) * math.exp(null[h].item() - taus[h])
                live = pos >= 0
                # a masked key's gate is not read, whatever it holds
                gz = torch.nan_to_num(g[:, h], nan=0.0, posinf=0.0, neginf=0.0)
                o[live, h] = (w[live] @ gz) / den[live, None]
                a[live, h] = (w[live] @ gz.abs()) / den[live, None]
                bad = ~torch.isfinite(g[:, h])
                for i, j in [(i, j) for i in range(n) for j in torch.where(bad.any(1))[0].tolist() if seen[i, j]]:
                    o[i, h] = torch.where(bad[j], g[j, h], o[i, h])
            out.append(o)
            mag.append(a)
            row += n
        o, a = torch.cat(out), torch.cat(mag)
        if v is not False:
            vv = (self.v if v is True else v).double().cpu().view(self.N, H, -1)[..., :self.m_h]
            o, a = o * vv, a * vv.abs()
        return o, a

    def check(self, **kw):
        tau_max = 10.0 if kw.get("tau") is None else kw["tau"].max().item()
        tau_max = kw.get("s", tau_max) if kw.get("tau") is None else tau_max
        got = self.run(**kw).double().cpu().view(self.N, self.H, -1)[..., :self.m_h]
        ok = {k: kw[k] for k in ("v", "tau", "s", "null") if k in kw}
        ok = {k: (x.cpu() if torch.is_tensor(x) and k != "v" else x) for k, x in ok.items()}
        want, mag = self.want(**ok)
        weight = tau_max * (self.d_h + 4) * 2.0 ** -23 + 2.0 ** -21 + (2.0 ** -8 if self.dtype == "bf16" else 0.0)
        tol = HALF_STEP[self.dtype] * 1.01 * want.abs() + (2 * weight + SUMS[self.dtype]) * mag + 1e-30
        fin = torch.isfinite(want)
        assert torch.equal(torch.isfinite(got), fin)
        worst = ((got - want).abs() / tol)[fin].max().item() if fin.any() else 0.0
        assert worst <= 1.0, worst
        st, word = tg.tg_check_device_error()
        assert st == tg.TG_OK, hex(word)
        return got


STEP = [(1, t) for t in (1, 2, 15, 16, 17, 64, 127, 128, 129, 300)]
FEW = [(3, 3), (8, 8), (5, 200), (1, 1), (2, 65), (7, 130), (0, 40), (8, 513)]
MID = [(64, 64), (33, 250), (100, 300), (9, 9), (17, 1000), (1, 700), (0, 5), (128, 128)]
CHUNK = [(130, 130), (1, 77), (0, 0), (64, 64), (33, 250), (9, 9), (129, 400), (17, 1000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,d_h,m_h,pitch,page", [(2, 64, 520, 520, 16), (4, 32, 252, 256, 64), (1, 16, 1100, 1104, 8),
                                                  (2, 64, 300, 304, 128)])
@pytest.mark.parametrize("seqs", [STEP, FEW, MID, CHUNK], ids=["step", "few", "mid", "chunk"])
def test_ragged(seqs, H, d_h, m_h, pitch, page, dtype):
    Batch(seqs, H, d_h, m_h, dtype, page, pitch).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seqs", [STEP, FEW, MID, CHUNK], ids=["step", "few", "mid", "chunk"])
def test_null_tau_and_no_v(seqs, dtype):
    """The null gate, per-head temperatures up to 20 and 0, gates alone."""
    b = Batch(seqs, 3, 32, 264, dtype, 32, seed=1)
    null = torch.tensor([0.5, -3.0, 8.0]).cuda()
    tau = torch.tensor([20.0, 0.0, 4.5]).cuda()
    b.check(null=null, tau=tau, v=False)
    b.check(null=null, s=20.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 3, 12, 100, 256])
def test_page_sizes(page, dtype):
    """Pages of any size: ends inside every tile."""
    Batch([(1, 50), (20, 333), (140, 300), (2, 2)], 2, 32, 136, dtype, page, seed=2).check()


@pytest.mark.parametrize("dtype,H,d_h,m_h,pitch", [("f32", 2, 48, 101, 101), ("f32", 3, 5, 33, 40), ("f32", 1, 128, 515, 515),
                                                   ("bf16", 2, 48, 77, 77), ("bf16", 2, 128, 130, 136)])
@pytest.mark.parametrize("seqs", [[(1, 70), (1, 1)], [(6, 90), (2, 20)], [(70, 170), (20, 20)]], ids=["step", "few", "chunk"])
def test_odd_widths(seqs, dtype, H, d_h, m_h, pitch):
    """Head widths and gate widths that no 16-byte vector divides."""
    Batch(seqs, H, d_h, m_h, dtype, 16, pitch, seed=3).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_context(dtype):
    """Long caches: spans joined from many parts; many rows against a long prefix."""
    Batch([(1, 5000), (1, 37)], 2, 64, 264, dtype, 64, seed=4).check()
    Batch([(40, 4100), (300, 2000)], 1, 64, 264, dtype, 64, seed=5).check()


@pytest.mark.parametrize("length", [449, 700, 769, 3000, 6200, 6209])
@pytest.mark.parametrize("n", [1, 20])
def test_key_ranges_cut_every_way(n, length):
    """Lengths whose steps divide evenly over the key ranges, and not: no range is empty and
    none is lost."""
    Batch([(n, length)], 1, 32, 72, "bf16", 32, seed=length).check()


def test_many_sequences():
    """More sequences than a warp's window of 32, some without new tokens, in one launch."""
    seqs = [((i * 7) % 4, 3 + (i * 37) % 190) for i in range(150)]
    Batch(seqs, 2, 16, 72, "bf16", 16, seed=40).check()
    Batch(seqs[:70] + [(90, 95)] + seqs[70:], 2, 16, 72, "bf16", 16, seed=41).check()
    Batch(seqs, 2, 16, 72, "f32", 16, seed=42).check()


def test_tiles_of_every_size_in_one_launch():
    """Several jobs per SM, tiles of one row and of 128 in turn, gates over many strips: what
    one tile leaves in shared memory must not reach the next."""
    seqs = [(300, 300), (1, 500), (7, 20), (129, 600), (1, 64), (16, 90), (17, 80), (1, 1), (200, 260), (2, 130)]
    b = Batch(seqs, 2, 32, 3500, "bf16", 32, 3504, seed=50)
    first = b.check()
    for _ in range(5):
        assert torch.equal(b.run().double().cpu().view(b.N, 2, -1)[..., :3500], first)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_without_keys(dtype):
    """Rows at negative positions see nothing: zeros, and the others are not touched."""
    b = Batch([(4, 2), (3, 0), (1, 9), (150, 140)], 2, 32, 128, dtype, 16, seed=6)
    b.check(null=torch.tensor([0.0, 1.0]).cuda())
    out = b.check()
    assert (out[:2] == 0).all() and (out[4:7] == 0).all() and (out[8:18] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [5, 40, 200])
def test_masked_gates_may_be_anything(n, dtype):
    """A NaN or infinite gate (or key) of a token reaches only the tokens that see it."""
    b = Batch([(n, n + 30), (n, n)], 2, 32, 264, dtype, 16, seed=7)
    j = 30 + n // 2            # a new token of the first sequence
    page, slot = b.table[0, j // 16].item(), j % 16
    for col, x in ((3, math.nan), (70, math.inf), (263, -math.inf)):
        b.gates[0][j, 1, col] = x
        b.g_pages[page, slot].view(2, -1)[1, col] = x
    out = b.check(v=False)
    assert torch.isfinite(out[:n // 2]).all() and torch.isfinite(out[n:]).all()
    assert not torch.isfinite(out[n // 2:n, 1, 3]).any()
    # the last new token's key: every other row is as it was
    j = 30 + n - 1
    b.k_pages[b.table[0, j // 16].item(), j % 16] = math.nan
    again = b.run(v=False).double().cpu().view(b.N, 2, -1)
    keep = [r for r in range(b.N) if r != n - 1]
    assert torch.equal(torch.nan_to_num(again[keep], nan=9e9), torch.nan_to_num(out[keep], nan=9e9))


def test_same_as_the_whole_sequence():
    """Chunk by chunk over the cache equals tango_aggregate's rows (fp32, and bf16 up to
    the weights' and outputs' roundings, both sides)."""
    for dtype in ("f32", "bf16"):
        T, H, d_h, m_h = 260, 2, 64, 256
        b = Batch([(T, T)], H, d_h, m_h, dtype, 16, seed=8)
        k = b.keys[0].reshape(1, T, -1).cuda()
        g = b.gates[0].reshape(1, T, -1).cuda()
        whole = torch.empty(1, T, H * m_h, dtype=DT[dtype], device="cuda")
        tg.tango_aggregate(b.q[None], k, g, b.v[None], whole, H=H, flags=tg.TG_FLAG_QK_NORMALIZED)
        for cuts in ([T], [200, 259, T], [1, 2, 3, 131, T]):
            a = 0
            for e in cuts:
                out = torch.empty(e - a, H * m_h, dtype=DT[dtype], device="cuda")
                cu = torch.tensor([0, e - a], dtype=torch.int32, device="cuda")
                ln = torch.tensor([e], dtype=torch.int32, device="cuda")
                tg.tango_paged_aggregate(b.q[a:e], b.v[a:e], out, b.k_pages, b.g_pages, b.table, cu, ln, H=H,
                                         max_new=e - a, max_len=e)
                d = (out.double() - whole[0, a:e].double()).abs().max().item()
                assert d <= (2e-5 if dtype == "f32" else 6 * 2.0 ** -8 * whole.abs().max().item())
                a = e


def test_slices_and_in_place():
    """v as a column slice of a wider tensor; out written over v."""
    for dtype, n in (("f32", 3), ("bf16", 3), ("bf16", 40)):
        b = Batch([(n, 50)], 2, 32, 128, dtype, 16, seed=9)
        wide = torch.randn(n, 512, device="cuda").to(DT[dtype])
        b.check(v=wide[:, 128:384])
        want = b.run()
        v = b.v.clone()
        tg.tango_paged_aggregate(b.q, v, v, b.k_pages, b.g_pages, b.table, b.cu, b.lens, H=2, max_new=n, max_len=50)
        assert torch.equal(v, want)


@pytest.mark.parametrize("n", [1, 12, 70])
def test_addresses_off_16_bytes(n):
    """v, q, out or a pool that start anywhere: other kernels, the same values."""
    b = Batch([(n, 90), (n, 300)], 2, 32, 264, "bf16", 16, seed=14)

    def off(t):
        x = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        x.copy_(t)
        return x
    b.check(v=torch.cat([b.v.new_zeros(b.N, 3), b.v], 1)[:, 3:])
    for name in ("q", "k_pages", "g_pages"):
        keep = getattr(b, name)
        setattr(b, name, off(keep))
        b.check()
        setattr(b, name, keep)
    out = off(torch.zeros(b.N, 528, dtype=torch.bfloat16, device="cuda"))
    tg.tango_paged_aggregate(b.q, b.v, out, b.k_pages, b.g_pages, b.table, b.cu, b.lens, H=2, max_new=n, max_len=300)
    assert (out.double() - b.run().double()).abs().max().item() <= 4 * 2.0 ** -8 * out.abs().max().item()


@pytest.mark.parametrize("dtype,n", [("bf16", 1), ("bf16", 20), ("f32", 3)])
def test_pages_beyond_32_bit_offsets(dtype, n):
    """Slots whose element offset passes 2^31: appended to and read back."""
    m_h, pages = 14240, 1250          # 1,250 pages x 64 tokens x 28,480 gates = 2.28e9 values
    b = Batch([(n, 70), (n, 130)], 2, 64, m_h, dtype, 64, seed=15)
    dt, first = DT[dtype], pages - b.k_pages.shape[0]
    k_pages = torch.empty(pages, 64, 128, dtype=dt, device="cuda")
    g_pages = torch.empty(pages, 64, 2 * m_h, dtype=dt, device="cuda")
    k_pages[first:], g_pages[first:] = b.k_pages, b.g_pages
    b.k_pages, b.g_pages, b.table = k_pages, g_pages, b.table + first
    assert first * 64 * 2 * m_h > 2 ** 31
    b.check()
    # the last tokens' gates once more, through the append
    k = torch.randn(b.N, 128, device="cuda").to(dt)
    g = torch.randn(b.N, 2 * m_h, device="cuda").to(dt)
    tg.tango_cache_append(None, k, g, None, k_pages, g_pages, b.table, b.cu, b.lens, None, H=2, norm=tg.TG_NORM_NONE,
                          silu=False)
    pos = torch.cat([torch.arange(t - n, t) for n, t in b.seqs]).cuda()
    seq = torch.arange(2).repeat_interleave(n).cuda()
    page = b.table[seq, pos // 64].long()
    assert torch.equal(g_pages[page, pos % 64], g) and torch.equal(k_pages[page, pos % 64], k)


@pytest.mark.parametrize("seed", range(24))
def test_seeded_draws(seed):
    """Head and gate widths, page sizes, lengths and options at random."""
    import random
    rng = random.Random(seed)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    H, d_h = rng.choice([(1, 64), (2, 64), (4, 32), (3, 16), (2, 128), (2, 24)])
    m_h = rng.randrange(1, 900)
    pitch = rng.choice([m_h, -(-m_h // 8) * 8, -(-m_h // 8) * 8 + 8])
    page = rng.choice([1, 5, 8, 16, 24, 32, 64, 96, 128, 256])
    most = rng.choice([1, 1, 8, 40, 300])
    seqs = []
    for _ in range(rng.randrange(1, 9)):
        new = rng.randrange(0, most + 1)
        seqs.append((new, rng.choice([new, new + rng.randrange(0, 70), new + rng.randrange(0, 900), max(0, new - 2)])))
    if not any(n for n, _ in seqs):
        seqs[0] = (1, 5)
    kw = dict(v=rng.choice([True, False]), s=rng.choice([0.0, 3.5, 10.0, 20.0]))
    if rng.random() < 0.4:
        kw["null"] = torch.randn(H, generator=torch.Generator().manual_seed(seed)).cuda()
    Batch(seqs, H, d_h, m_h, dtype, page, pitch, seed=seed).check(**kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeats_bit_for_bit(dtype):
    """Joined spans add in a fixed order; a workspace's earlier contents do not matter."""
    for seqs in ([(1, 3000), (1, 700)], [(200, 2100), (3, 900)]):
        b = Batch(seqs, 2, 64, 520, dtype, 64, seed=10)
        outs = []
        for fill in (0, 255, 127):
            p = tg.paged_params(b.N, b.k_pages, b.g_pages, b.table, b.cu, b.lens, H=2, max_new=b.max_new,
                                max_len=b.max_len, m_h=520)
            ws = torch.full((tg.tg_workspace_size(tg.TG_WS_PAGED, p) + 256,), fill, dtype=torch.uint8, device="cuda")
            outs.append(b.run(ws=ws))
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_bounds_looser_than_the_batch():
    """max_new and max_len are upper bounds only."""
    for dtype in ("bf16", "f32"):
        b = Batch([(1, 40), (1, 3)], 2, 32, 128, dtype, 16, seed=11)
        b.table = torch.cat([b.table, b.table.new_full((2, 60), -1)], 1).contiguous()
        a = b.check()
        for new, length in ((2, 64), (9, 900), (300, 1000)):
            b.check(max_new=new, max_len=length)
        assert a is not None


def test_side_stream_and_graph():
    """On another stream, and captured once and replayed for later steps of the lengths."""
    for n in (1, 20):
        b = Batch([(n, 90), (n, 300)], 2, 32, 264, "bf16", 16, seed=12)
        want = b.run()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        out = torch.zeros_like(want)
        call = lambda: tg.tango_paged_aggregate(b.q, b.v, out, b.k_pages, b.g_pages, b.table, b.cu, b.lens, H=2,  # noqa: E731
                                                max_new=n, max_len=300, m_h=264)
        with torch.cuda.stream(s):
            call()
        s.synchronize()
        assert torch.equal(out, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
        b.lens.copy_(torch.tensor([70, 299], dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, b.run())


@pytest.mark.parametrize("seqs", [[(1, 3000)], [(2, 2500), (1, 1025)], [(4, 1100), (3, 1024)], [(8, 2100), (5, 1089)]])
def test_sums_of_many_key_spans_are_joined_in_order(seqs):
    """More than 16 spans of one output (groups of spans, then the groups), full tiles and
    tiles with rows to spare, on the CUDA cores in both types; the same bits every time."""
    for dtype, pitch in (("f32", 260), ("f32", 259), ("bf16", 259)):
        b = Batch(seqs, 2, 16, 259, dtype, 16, pitch=pitch, seed=21)
        got = b.check()
        for _ in range(3):
            assert torch.equal(b.run().double().cpu().view(b.N, 2, -1)[..., :259], got)


def test_scratch_is_taken_from_the_calls_stream(monkeypatch):
    """A call on a stream that is not the current one allocates its scratch there: a block
    freed on the current stream may still be written by work that waits on it."""
    b = Batch([(20, 90), (20, 300)], 2, 32, 264, "bf16", 16, seed=12)
    want, out = b.run(), torch.zeros(b.N, 2 * 264, dtype=torch.bfloat16, device="cuda")
    x, dx, gain = torch.randn(40, 64, device="cuda"), torch.empty(40, 64, device="cuda"), torch.ones(32, device="cuda")
    torch.cuda.synchronize()
    took, allocate = [], tg._workspace
    monkeypatch.setattr(tg, "_workspace",
                        lambda *a: (took.append(torch.cuda.current_stream().cuda_stream), allocate(*a))[1])
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    for stream in (side, side.cuda_stream, 0, None):
        out.zero_()
        torch.cuda.synchronize()
        tg.tango_paged_aggregate(b.q, b.v, out, b.k_pages, b.g_pages, b.table, b.cu, b.lens, H=2, max_new=20,
                                 max_len=300, m_h=264, stream=stream)
        tg.tango_qk_norm_rope_backward(x, None, x, None, dx, None, None, H=2, norm=tg.TG_NORM_RMS, q_gain=gain,
                                       dq_gain=torch.empty_like(gain), stream=stream)
        where = here.cuda_stream if stream is None else getattr(stream, "cuda_stream", stream)
        assert took == [where, where]
        assert torch.cuda.current_stream() == here
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        took.clear()


def test_bad_device_values_are_flagged_and_not_followed():
    """Pages outside the pool, lengths and row offsets outside their bounds: the checks in
    the kernels skip or clamp them and set the error word."""
    for n in (1, 6, 40):
        for what in ("page", "len", "cu"):
            b = Batch([(n, 60), (n, 200)], 2, 32, 264, "bf16", 16, seed=13)
            if what == "page":
                b.table[1, 2] = 10 ** 6
            elif what == "len":
                b.lens[1] = 10 ** 8
            else:
                b.cu[1] = 10 ** 7
            b.run()
            st, word = tg.tg_check_device_error()
            assert st == tg.TG_ERR_DEVICE and (word >> 8) & 0xff == 6
            assert tg.tg_check_device_error()[0] == tg.TG_OK


# ------------------------------------------------------------------------------ append

def _turned(x, d_h, pos, freqs, layout):
    x = x.double().cpu().reshape(x.shape[0], -1, d_h)
    z = x / x.norm(dim=-1, keepdim=True).clamp(min=1e-12)
    r = 2 * freqs.numel()
    ang = pos.double()[:, None] * freqs.double().cpu()
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    i = torch.arange(r // 2)
    a, b = (i, i + r // 2) if layout == tg.TG_ROPE_HALF else (2 * i, 2 * i + 1)
    p, q = z[..., a].clone(), z[..., b].clone()
    z[..., a], z[..., b] = p * c - q * s, p * s + q * c
    return z.flatten(1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,d_h,m_h,pitch,page,rotary,layout", [
    (2, 64, 520, 520, 16, 64, 0), (16, 32, 60, 64, 64, 32, 1), (2, 64, 77, 77, 5, 48, 0), (1, 20, 1100, 1104, 8, 6, 1)])
def test_append(H, d_h, m_h, pitch, page, rotary, layout, dtype):
    seqs = [(1, 1), (1, 40), (17, 17), (5, 100), (0, 30), (3, 2), (90, 200)]
    b = Batch(seqs, H, d_h, m_h, dtype, page, pitch, seed=20, fill=False)
    g = torch.Generator().manual_seed(21)
    dt = DT[dtype]
    wide = (3 * torch.randn(b.N, 2 * H * d_h + H * pitch + 16, generator=g)).to(dt).cuda()
    q, k = wide[:, :H * d_h], wide[:, H * d_h:2 * H * d_h].contiguous()
    gates = (3 * torch.randn(b.N, H * pitch, generator=g)).to(dt).cuda()
    fr = tg.tg_rope_freqs(rotary, factor=4.0)
    for silu in (True, False):
        kp, gp = torch.full_like(b.k_pages, math.nan), torch.full_like(b.g_pages, math.nan)
        qo = torch.empty(b.N, H * d_h, dtype=dt, device="cuda")
        tg.tango_cache_append(q, k, gates, qo, kp, gp, b.table, b.cu, b.lens, fr, H=H, m_h=m_h, layout=layout, silu=silu)
        assert tg.tg_check_device_error()[0] == tg.TG_OK
        pos = torch.cat([torch.arange(t - n, t) for n, t in seqs])
        seq = torch.cat([torch.full((n,), i) for i, (n, _) in enumerate(seqs)])
        live = pos >= 0
        table = b.table.cpu()
        at = torch.zeros(b.N, dtype=torch.long)
        at[live] = table[seq[live], pos[live] // page].long() * page + pos[live] % page
        for got, src in ((qo.cpu()[live], q), (kp.cpu().reshape(-1, H * d_h)[at[live]], k)):
            want = _turned(src, d_h, pos, fr, layout)[live]
            tol = HALF_STEP[dtype] * want.abs() * 1.001 + (d_h / 2 + 12) * 2.0 ** -24 + 2.0 ** -22
            assert ((got.double() - want).abs() / tol).max().item() <= 1.0
        x = gates.double().cpu().view(b.N, H, pitch)[..., :m_h][live]
        want = x * torch.sigmoid(x) if silu else x
        got = gp.cpu().reshape(-1, H, pitch)[at[live]][..., :m_h].double()
        # SiLU in fp32: the exponential's and the quotient's few 2^-21, and the rounding
        tol = HALF_STEP[dtype] * want.abs() * 1.001 + 2.0 ** -20 * want.abs() + 1e-30 if silu else torch.full_like(want, 1e-300)
        assert ((got - want).abs() / tol).max().item() <= 1.0
        # every other slot is as it was
        rest = torch.ones(kp.shape[0] * page, dtype=torch.bool)
        rest[at[live]] = False
        assert torch.isnan(kp.cpu().reshape(-1, H * d_h)[rest]).all()
        assert torch.isnan(gp.cpu().reshape(-1, H * pitch)[rest]).all()


def test_append_flags_bad_values():
    for what in ("page", "len", "cu"):
        b = Batch([(2, 60), (3, 200)], 2, 32, 264, "bf16", 16, seed=22)
        k, g = torch.randn(5, 64, device="cuda").bfloat16(), torch.randn(5, 528, device="cuda").bfloat16()
        if what == "page":
            b.table[1, 12] = -3
        elif what == "len":
            b.lens[1] = 10 ** 8
        else:
            b.cu[1] = -9
        tg.tango_cache_append(None, k, g, None, b.k_pages, b.g_pages, b.table, b.cu, b.lens, tg.tg_rope_freqs(32), H=2)
        st, word = tg.tg_check_device_error()
        assert st == tg.TG_ERR_DEVICE and (word >> 8) & 0xff == 6


def test_append_then_aggregate_equals_the_whole_sequence():
    """Token by token and chunk by chunk through append and aggregate, against the library's
    own whole-sequence path on raw q, k and gates (fp32: both sides a few 2^-20)."""
    T, H, d_h, m_h, page = 45, 2, 64, 200, 8
    g = torch.Generator().manual_seed(30)
    q, k = torch.randn(T, H * d_h, generator=g).cuda(), torch.randn(T, H * d_h, generator=g).cuda()
    raw, v = torch.randn(T, H * m_h, generator=g).cuda(), torch.randn(T, H * m_h, generator=g).cuda()
    fr = tg.tg_rope_freqs(d_h)
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    tg.tango_qk_norm_rope(q, k, qr, kr, fr, H=H)
    whole = torch.empty(1, T, H * m_h, device="cuda")
    tg.tango_aggregate(qr[None], kr[None], torch.nn.functional.silu(raw)[None], v[None], whole, H=H)
    kp, gp = tg.cache_pools(6, page, H, d_h, m_h, dtype=torch.float32)
    table = torch.tensor([[4, 0, 5, 2, 1, 3]], dtype=torch.int32, device="cuda")
    a = 0
    for e in [7, 8, 9, 30] + list(range(31, T + 1)):
        cu = torch.tensor([0, e - a], dtype=torch.int32, device="cuda")
        ln = torch.tensor([e], dtype=torch.int32, device="cuda")
        qo, out = torch.empty(e - a, H * d_h, device="cuda"), torch.empty(e - a, H * m_h, device="cuda")
        tg.tango_cache_append(q[a:e], k[a:e], raw[a:e], qo, kp, gp, table, cu, ln, fr, H=H)
        tg.tango_paged_aggregate(qo, v[a:e], out, kp, gp, table, cu, ln, H=H, max_new=e - a, max_len=T)
        assert (out - whole[0, a:e]).abs().max().item() <= 2e-5 * whole.abs().max().item()
        a = e


# ------------------------------------------------------------------------------ passes

PASSES = [(130, 300), (1, 700), (40, 41), (0, 9), (64, 600), (60, 60)]  # 295 rows


def _loose(b, max_len):
    """The batch with a page table that a bound of max_len tokens needs, and its scratch with
    H heads."""
    b.table = torch.cat([b.table, b.table.new_full((b.B, -(-max_len // b.page)), -1)], 1).contiguous()

    def scratch(H):
        p = tg.paged_params(b.N, b.k_pages, b.g_pages, b.table, b.cu, b.lens, H=b.H, max_new=b.max_new, max_len=max_len,
                            m_h=b.m_h)
        p.m, p.H = p.m // p.H * H, H
        return tg.tg_workspace_size(tg.TG_WS_PAGED, p)
    return scratch


@pytest.mark.parametrize("dtype,d_h", [("f32", 32), ("bf16", 128)])
def test_cuda_core_passes_over_heads_and_tiles(dtype, d_h):
    """Bounds far above the batch make one pass's scratch too small for all heads, then for all
    tiles of one head; the last pass of either kind is a shorter one."""
    for max_len, by_tiles in ((1 << 17, False), (900000, True)):
        b = Batch(PASSES, 7, d_h, 72, dtype, 64, seed=60)
        scratch = _loose(b, max_len)
        assert scratch(7) <= (1 << 30) + (1 << 16)
        # one head at a time; or several, but not all
        assert (scratch(7) == scratch(1)) == by_tiles and scratch(7) < 6 * scratch(1)
        null = torch.linspace(-1, 2, 7).cuda()
        got = b.check(null=null, max_len=max_len)
        assert torch.equal(b.run(null=null, max_len=max_len).double().cpu().view(b.N, 7, -1), got)


@pytest.mark.parametrize("seqs,max_len,cut", [
    (PASSES, 1 << 20, "heads"),                                             # 2 heads a pass, 7 in all
    (PASSES + [(300, 420), (200, 200)], 1 << 21, "rows"),                   # 384 rows a pass
    (PASSES, 1 << 23, "rows"),                                              # 128, the least
    ([(1 + i % 8, 20 + 3 * i) for i in range(110)], 1 << 21, "rows"),       # single tokens and a few
], ids=["heads", "rows", "least", "few"])
def test_tensor_core_passes_over_heads_and_rows(seqs, max_len, cut):
    """The same on the tensor cores, whose passes share the weights, denominators, partial sums
    and counters: by heads, and by tiles of one head where its weights alone pass 2 GB."""
    b = Batch(seqs, 7, 32, 72, "bf16", 64, seed=61)
    scratch = _loose(b, max_len)
    assert scratch(7) <= 5 << 30
    assert (scratch(7) == scratch(1)) == (cut == "rows") and scratch(7) < 6 * scratch(1)
    null = torch.linspace(-1, 2, 7).cuda()
    got = b.check(null=null, max_len=max_len)
    assert torch.equal(b.run(null=null, max_len=max_len).double().cpu().view(b.N, 7, -1), got)
    # one pass over all of it: the same weights, summed in other ranges, each rounded once
    assert (got - b.run(null=null).double().cpu().view(b.N, 7, -1)).abs().max().item() <= 2.0 ** -6 * got.abs().max().item()


def test_passes_of_unaligned_calls():
    """bf16 rows off 16 bytes take the CUDA cores in the scratch that the tensor cores would
    need: more passes, the same values."""
    b = Batch(PASSES, 7, 32, 72, "bf16", 64, seed=62)
    scratch = _loose(b, 1 << 17)
    assert scratch(7) < 1 << 30
    x = torch.empty(b.q.numel() + 1, dtype=b.q.dtype, device="cuda")[1:].view(b.q.shape)
    b.q = x.copy_(b.q)
    null = torch.linspace(-1, 2, 7).cuda()
    got = b.check(null=null, max_len=1 << 17)
    assert torch.equal(b.run(null=null, max_len=1 << 17).double().cpu().view(b.N, 7, -1), got)


@pytest.mark.parametrize("d_h", [32, 20])
def test_appended_keys_keep_their_nan(d_h):
    """A key with one NaN is cached as NaN throughout its head, not as finite values without a
    meaning."""
    b = Batch([(3, 7)], 2, d_h, 40, "bf16", 8, seed=63, fill=False)
    k, g = torch.randn(3, 2 * d_h, device="cuda").bfloat16(), torch.randn(3, 80, device="cuda").bfloat16()
    k[1, d_h + 3] = math.nan
    b.k_pages.zero_()
    tg.tango_cache_append(None, k, g, None, b.k_pages, b.g_pages, b.table, b.cu, b.lens, None, H=2)
    got = b.k_pages[b.table[0, 0].item(), 4:7].view(3, 2, d_h)
    assert got[1, 1].isnan().all() and torch.isfinite(got[[0, 2]]).all() and torch.isfinite(got[1, 0]).all()


# ------------------------------------------------------------------------- unit vectors

@pytest.mark.parametrize("dtype,d_h", [("bf16", 64), ("f32", 64), ("bf16", 48)])
@pytest.mark.parametrize("n", [1, 6, 40])
def test_vectors_that_are_not_unit_are_flagged(n, dtype, d_h):
    """RMS-normed keys and queries have products up to d_h: weights beyond fp32.  The call says so
    instead of returning what is left of them."""
    b = Batch([(n, 60), (n, 200)], 2, d_h, 264, dtype, 16, seed=64)
    k = torch.randn(b.N, 2 * d_h, device="cuda").to(DT[dtype])
    g, qo = torch.randn(b.N, 528, device="cuda").to(DT[dtype]), torch.empty_like(k)
    how = dict(page_table=b.table, cu_new=b.cu, lens=b.lens, H=2)
    for norm, status in ((tg.TG_NORM_UNIT, tg.TG_OK), (tg.TG_NORM_RMS, tg.TG_ERR_DEVICE), (tg.TG_NORM_UNIT, tg.TG_OK)):
        # (a token's own key is its query here: their product is d_h)
        tg.tango_cache_append(k, k, g, qo, b.k_pages, b.g_pages, freqs=None, norm=norm, **how)
        b.q = qo
        b.run()
        st, word = tg.tg_check_device_error()
        assert st == status and (st == tg.TG_OK or ((word >> 8) & 0xff == 6 and word & 2))
    # the other way: products of -64, whose weights vanish
    b.k_pages[:] = -qo[0]
    b.q = (64 * qo[:1]).expand(b.N, -1).contiguous()
    b.run()
    assert tg.tg_check_device_error()[0] == tg.TG_ERR_DEVICE


def test_extreme_unit_vectors_are_not_flagged():
    """Keys equal and opposite to the query at tau = 20, and zero vectors, with components rounded
    away from zero, stay inside the range."""
    for dtype in ("bf16", "f32"):
        for n in (1, 6, 40):
            b = Batch([(n, 130)], 1, 64, 72, dtype, 16, seed=65)
            # half of the components one step up: 1 + 2^-8 long, as far as bf16 rounding goes
            x = torch.full((64,), 0.125)
            x[::2] *= 1 + 2.0 ** -7
            for sign in (1.0, -1.0, 0.0):
                b.q = x.to(DT[dtype]).repeat(n, 1).cuda()
                b.keys[0] = (sign * x).to(DT[dtype]).view(1, 1, 64).repeat(130, 1, 1)
                for p in range(b.table.shape[1] - 1):
                    b.k_pages[b.table[0, p].item()] = b.keys[0][0].cuda()
                b.run(s=20.0)
                assert tg.tg_check_device_error()[0] == tg.TG_OK


def test_training_with_gains_serves_through_the_cache():
    """RMS norm with gains, rotation, then the aggregation's own unit norm, as training has it:
    served by tango_qk_norm_rope at the tokens' positions and an append that makes unit vectors
    (fp32: both sides a few 2^-20)."""
    T, H, d_h, m_h = 70, 2, 64, 200
    g = torch.Generator().manual_seed(66)
    q, k = torch.randn(T, H * d_h, generator=g).cuda(), torch.randn(T, H * d_h, generator=g).cuda()
    gates, v = torch.randn(T, H * m_h, generator=g).cuda(), torch.randn(T, H * m_h, generator=g).cuda()
    how = dict(H=H, norm=tg.TG_NORM_RMS, q_gain=(1 + 0.3 * torch.randn(d_h, generator=g)).cuda(),
               k_gain=(1 + 0.3 * torch.randn(d_h, generator=g)).cuda())
    fr = tg.tg_rope_freqs(d_h)
    qr, kr, whole = torch.empty_like(q), torch.empty_like(k), torch.empty(1, T, H * m_h, device="cuda")
    tg.tango_qk_norm_rope(q, k, qr, kr, fr, **how)
    tg.tango_aggregate(qr[None], kr[None], gates[None], v[None], whole, H=H)
    kp, gp = tg.cache_pools(5, 16, H, d_h, m_h, dtype=torch.float32)
    table = torch.tensor([[3, 0, 4, 1, 2]], dtype=torch.int32, device="cuda")
    a = 0
    for e in (33, 34, 50, T):
        cu, ln = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, e - a], [e]))
        pos = torch.arange(a, e, dtype=torch.int32, device="cuda")
        qa, ka, qo = (torch.empty(e - a, H * d_h, device="cuda") for _ in range(3))
        out = torch.empty(e - a, H * m_h, device="cuda")
        tg.tango_qk_norm_rope(q[a:e], k[a:e], qa, ka, fr, positions=pos, **how)
        tg.tango_cache_append(qa, ka, gates[a:e], qo, kp, gp, table, cu, ln, None, H=H, silu=False)
        tg.tango_paged_aggregate(qo, v[a:e], out, kp, gp, table, cu, ln, H=H, max_new=e - a, max_len=T)
        assert (out - whole[0, a:e]).abs().max().item() <= 2e-5 * whole.abs().max().item()
        a = e
    assert tg.tg_check_device_error()[0] == tg.TG_OK


@pytest.mark.parametrize("seqs", [[(1, 70), (1, 1300)], [(40, 300), (200, 260), (1, 5)], [(600, 2000)]],
                         ids=["few", "chunks", "ranges"])
def test_bounded_wait_timeout_reports_status(seqs):
    """TG_FLAG_DEBUG_TIMEOUT makes the tensor-core kernels wait on barriers that nothing signals:
    the waits run out after 1 ms, every role leaves its loops, copies in flight are waited for,
    and the error word says so.  The next call is right."""
    b = Batch(seqs, 2, 32, 520, "bf16", 16, seed=67)
    b.run(flags=tg.TG_FLAG_DEBUG_TIMEOUT)
    st, word = tg.tg_check_device_error()
    assert st == tg.TG_ERR_TIMEOUT and word & 1 and (word >> 8) & 0xff == 6
    assert tg.tg_check_device_error() == (tg.TG_OK, 0)
    first = b.check()
    assert torch.equal(b.run().double().cpu().view(b.N, 2, -1), first)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 40])
def test_rows_of_no_sequence_are_left_alone(n, dtype):
    """Rows before cu_new[0] and from cu_new[B] on (a captured graph's spare rows) keep what they
    hold, whatever q and v hold there; the others are as without them."""
    b = Batch([(n, 60), (n, 200)], 2, 32, 264, dtype, 16, seed=68)
    want = b.run()

    def padded(t, fill):
        spare = torch.full_like(t[:1], fill)
        return torch.cat([spare.repeat(3, 1), t, spare.repeat(150, 1)])
    b.q, b.v, b.cu, out = padded(b.q, math.nan), padded(b.v, math.nan), b.cu + 3, padded(torch.zeros_like(want), 7.0)
    tg.tango_paged_aggregate(b.q, b.v, out, b.k_pages, b.g_pages, b.table, b.cu, b.lens, H=2, max_new=n, max_len=200)
    assert torch.equal(out[3:3 + b.N], want)
    assert (out[:3] == 7).all() and (out[3 + b.N:] == 7).all()
    k, g = padded(b.q[3:3 + b.N], 1.0), padded(b.v[3:3 + b.N], 1.0)
    kp, gp = torch.full_like(b.k_pages, math.nan), torch.full_like(b.g_pages, math.nan)
    tg.tango_cache_append(None, k, g, None, kp, gp, b.table, b.cu, b.lens, None, H=2)
    assert torch.isfinite(kp[..., 0]).sum() == b.N and torch.isfinite(gp[..., 0]).sum() == b.N
    assert tg.tg_check_device_error()[0] == tg.TG_OK
