"""Host-side checks of the norm-and-rotate calls and the paged cache calls: bad arguments
are refused before anything is launched, on a machine without a GPU too."""
import ctypes
import math

import pytest
import torch

import cross_token_gated_gb300 as tg

A = 256  # a pointer that validation never follows


def _qk(**kw):
    base = dict(rows=4, H=2, H_k=2, d_h=64, rotary_dim=64, layout=0, norm=1, eps=1e-6, T=4, positions=None, freqs=A,
                q_gain=None, k_gain=None, q_pitch=0, k_pitch=0, dtype=tg.TG_BF16)
    base.update(kw)
    return tg.tg_qk_params(*base.values())


def _paged(**kw):
    base = dict(B=2, H=2, d_h=64, m=512, m_pitch=0, N=3, max_new=2, max_len=40, page_size=16, n_pages=8, table_pitch=4,
                cu_new=A, lens=A, page_table=A, s=10.0, tau=None, null_bias=None, v_pitch=0, dtype=tg.TG_BF16)
    base.update(kw)
    return tg.tg_paged_params(*base.values())


def _append(**kw):
    base = dict(rotary_dim=64, layout=0, norm=1, eps=1e-6, freqs=A, silu=1, q_pitch=0, k_pitch=0, g_pitch=0)
    base.update(kw)
    return tg.tg_append_params(*base.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), tg.TG_ERR_INVALID_ARG),
    (dict(H=0), tg.TG_ERR_INVALID_ARG),
    (dict(H_k=-1), tg.TG_ERR_INVALID_ARG),
    (dict(d_h=0), tg.TG_ERR_INVALID_ARG),
    (dict(rotary_dim=63), tg.TG_ERR_INVALID_ARG),
    (dict(rotary_dim=66), tg.TG_ERR_INVALID_ARG),
    (dict(freqs=None), tg.TG_ERR_INVALID_ARG),
    (dict(layout=2), tg.TG_ERR_INVALID_ARG),
    (dict(norm=3), tg.TG_ERR_INVALID_ARG),
    (dict(norm=tg.TG_NORM_RMS, eps=0.0), tg.TG_ERR_INVALID_ARG),
    (dict(T=0), tg.TG_ERR_INVALID_ARG),
    (dict(q_pitch=127), tg.TG_ERR_INVALID_ARG),
    (dict(k_pitch=127), tg.TG_ERR_INVALID_ARG),
    (dict(dtype=2), tg.TG_ERR_INVALID_ARG),
    (dict(d_h=130, rotary_dim=0), tg.TG_ERR_UNSUPPORTED),
])
def test_qk_refusals(lib, kw, status):
    raw, p = tg.load(), _qk(**kw)
    assert raw.tango_qk_norm_rope(ctypes.byref(p), A, A, A, A, None) == status
    assert raw.tango_qk_norm_rope_backward(ctypes.byref(p), A, A, A, A, A, A, None, None, None, 0, None) == status
    p.q_gain = A
    assert tg.tg_workspace_size(tg.TG_WS_QK_BWD, p) == 0


def test_qk_pointer_refusals(lib):
    raw, p = tg.load(), _qk()
    f, b = raw.tango_qk_norm_rope, raw.tango_qk_norm_rope_backward
    bad = tg.TG_ERR_INVALID_ARG
    assert f(None, A, A, A, A, None) == bad
    assert f(ctypes.byref(p), None, A, A, A, None) == bad
    assert f(ctypes.byref(p), A, None, A, A, None) == bad          # H_k = 2 needs k
    assert f(ctypes.byref(_qk(H_k=0)), A, A, A, A, None) == bad    # and no k where it is 0
    assert f(ctypes.byref(p), A + 1, A, A, A, None) == tg.TG_ERR_UNSUPPORTED
    assert b(ctypes.byref(p), A, A, A, A, A, A, A, None, None, 0, None) == bad    # dq_gain without a gain
    g = _qk(q_gain=A, k_gain=A)
    assert b(ctypes.byref(g), A, A, A, A, A, A, A, A, None, 0, None) == tg.TG_ERR_WORKSPACE
    assert tg.tg_workspace_size(tg.TG_WS_QK_BWD, p) == 0
    assert f(ctypes.byref(_qk(rows=0)), A, A, A, A, None) == tg.TG_OK           # nothing to do


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), tg.TG_ERR_INVALID_ARG),
    (dict(H=65), tg.TG_ERR_INVALID_ARG),
    (dict(m=511), tg.TG_ERR_INVALID_ARG),
    (dict(m_pitch=255), tg.TG_ERR_INVALID_ARG),
    (dict(N=-1), tg.TG_ERR_INVALID_ARG),
    (dict(max_new=0), tg.TG_ERR_INVALID_ARG),
    (dict(max_len=0), tg.TG_ERR_INVALID_ARG),
    (dict(max_len=65), tg.TG_ERR_INVALID_ARG),   # more than the table's pages hold
    (dict(page_size=0), tg.TG_ERR_INVALID_ARG),
    (dict(n_pages=0), tg.TG_ERR_INVALID_ARG),
    (dict(table_pitch=0), tg.TG_ERR_INVALID_ARG),
    (dict(cu_new=None), tg.TG_ERR_INVALID_ARG),
    (dict(lens=None), tg.TG_ERR_INVALID_ARG),
    (dict(page_table=None), tg.TG_ERR_INVALID_ARG),
    (dict(s=21.0), tg.TG_ERR_INVALID_ARG),
    (dict(s=math.nan), tg.TG_ERR_INVALID_ARG),
    (dict(v_pitch=511), tg.TG_ERR_INVALID_ARG),
    (dict(dtype=7), tg.TG_ERR_INVALID_ARG),
    (dict(d_h=129), tg.TG_ERR_UNSUPPORTED),
    (dict(page_size=1 << 17), tg.TG_ERR_UNSUPPORTED),
    (dict(n_pages=1 << 28), tg.TG_ERR_UNSUPPORTED),   # slot numbers pass 31 bits
])
def test_paged_refusals(lib, kw, status):
    raw, p, a = tg.load(), _paged(**kw), _append()
    if kw.get("d_h") == 129:
        a = _append(rotary_dim=0)
    assert raw.tango_paged_aggregate(ctypes.byref(p), A, A, A, A, A, None, 0, None) == status
    assert raw.tango_cache_append(ctypes.byref(p), ctypes.byref(a), A, A, A, A, A, A, None) == status
    assert tg.tg_workspace_size(tg.TG_WS_PAGED, p) == 0


def test_paged_pointer_refusals(lib):
    raw, p, a = tg.load(), _paged(), _append()
    P, bad = ctypes.byref, tg.TG_ERR_INVALID_ARG
    agg, app = raw.tango_paged_aggregate, raw.tango_cache_append
    assert agg(None, A, A, A, A, A, None, 0, None) == bad
    for i in (0, 2, 3, 4):
        args = [A] * 5
        args[i] = None
        assert agg(P(p), *args, None, 0, None) == bad
    assert agg(P(p), A, A + 1, A, A, A, None, 0, None) == tg.TG_ERR_UNSUPPORTED
    need = tg.tg_workspace_size(tg.TG_WS_PAGED, p)
    assert need > 0
    assert agg(P(p), A, A, A, A, A, None, 0, None) == tg.TG_ERR_WORKSPACE
    assert agg(P(p), A, A, A, A, A, 4096, need - 1, None) == tg.TG_ERR_WORKSPACE
    assert agg(P(p), A, A, A, A, A, 4096 + 16, need, None) == tg.TG_ERR_WORKSPACE
    assert agg(P(_paged(N=0)), A, A, A, A, A, None, 0, None) == tg.TG_OK
    assert app(P(p), None, A, A, A, A, A, A, None) == bad
    assert app(P(p), P(a), A, A, A, None, A, A, None) == bad       # q without q_out
    for i in (1, 2, 4, 5):
        args = [A] * 6
        args[i] = None
        assert app(P(p), P(a), *args, None) == bad
    for kw in (dict(rotary_dim=65), dict(rotary_dim=66), dict(freqs=None), dict(layout=5), dict(norm=9),
               dict(k_pitch=127), dict(q_pitch=127), dict(g_pitch=511)):
        assert app(P(p), P(_append(**kw)), A, A, A, A, A, A, None) == bad
    assert app(P(_paged(N=0)), P(a), A, A, A, A, A, A, None) == tg.TG_OK


def test_paged_workspace_grows_with_the_batch(lib):
    small = tg.tg_workspace_size(tg.TG_WS_PAGED, _paged())
    assert tg.tg_workspace_size(tg.TG_WS_PAGED, _paged(N=0)) == 0
    assert tg.tg_workspace_size(tg.TG_WS_PAGED, _paged(B=64, N=64, max_new=1)) > small


def test_rope_freqs(lib):
    """Base frequencies; all interpolated; and, with a trained length, fast pairs kept, slow
    ones interpolated, a linear ramp of turns between."""
    f = tg.tg_rope_freqs(64, device="cpu")
    want = torch.tensor([10000.0 ** (-2 * c / 64) for c in range(32)], dtype=torch.float64)
    assert torch.allclose(f, want, rtol=1e-15, atol=0)
    assert torch.allclose(tg.tg_rope_freqs(64, factor=8.0, device="cpu"), want / 8, rtol=1e-15, atol=0)
    g = tg.tg_rope_freqs(64, factor=8.0, orig_len=8192, turns_lo=1.0, turns_hi=4.0, device="cpu")
    turns = 8192 * want / (2 * math.pi)
    w = ((turns - 1) / 3).clamp(0, 1)
    assert torch.allclose(g, want * (w + (1 - w) / 8), rtol=1e-14, atol=0)
    assert (w == 1).any() and (w == 0).any() and ((w > 0) & (w < 1)).any()
    assert tg.tg_rope_freqs(0, device="cpu").numel() == 0
    for bad in (dict(base=0.0), dict(factor=0.5), dict(orig_len=-1), dict(orig_len=64, turns_lo=2.0, turns_hi=2.0),
                dict(factor=math.nan)):
        with pytest.raises(tg.TgError):
            tg.tg_rope_freqs(64, device="cpu", **bad)
    with pytest.raises(tg.TgError):
        tg.tg_rope_freqs(7, device="cpu")


def test_binding_checks_tensors(lib):
    """The binding refuses tensors the library would read as something else."""
    bf = torch.bfloat16
    q = torch.zeros(4, 128, dtype=bf)
    o = torch.zeros(4, 128, dtype=bf)
    fr = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(TypeError):
        tg.tango_qk_norm_rope(q, None, o.float(), None, fr, H=2)
    with pytest.raises(TypeError):
        tg.tango_qk_norm_rope(q, None, o, None, fr.float(), H=2)
    with pytest.raises(ValueError):
        tg.tango_qk_norm_rope(q.t(), None, o.t(), None, fr, H=2)          # columns not adjacent
    with pytest.raises(ValueError):
        tg.tango_qk_norm_rope(q, None, torch.zeros(4, 256, dtype=bf)[:, :128], None, fr, H=2)   # output not dense
    with pytest.raises(ValueError):
        tg.tango_qk_norm_rope(q, q[:2], o, o[:2], fr, H=2)
    with pytest.raises(ValueError):
        tg.tango_qk_norm_rope(q, None, o, None, fr, H=2, positions=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        tg.tango_qk_norm_rope(q[:1].expand(4, 128), None, o, None, fr, H=2)  # rows at pitch 0
    kp, gp = tg.cache_pools(4, 16, 2, 64, 100, device="cpu")
    assert gp.shape == (4, 16, 2 * 104)
    ints = dict(dtype=torch.int32)
    ok = dict(page_table=torch.zeros(1, 2, **ints), cu_new=torch.zeros(2, **ints), lens=torch.zeros(1, **ints))
    out = torch.zeros(4, 208, dtype=bf)
    kw = dict(H=2, max_new=4, max_len=32)
    with pytest.raises(TypeError):
        tg.tango_paged_aggregate(q, None, out, kp, gp, **dict(ok, lens=torch.zeros(1)), **kw)
    with pytest.raises(ValueError):
        tg.tango_paged_aggregate(q, None, out, kp, gp, **dict(ok, cu_new=torch.zeros(1, **ints)), **kw)
    with pytest.raises(ValueError):
        tg.tango_paged_aggregate(q, None, out[:3], kp, gp, **ok, **kw)
    with pytest.raises(ValueError):
        tg.tango_cache_append(None, q, out, q, kp, gp, **ok, freqs=fr, H=2)
    with pytest.raises(ValueError):
        tg.tango_cache_append(None, q, out[:, :200], None, kp, gp, **ok, freqs=fr, H=2)


def _cpu_calls():
    """Well-formed calls of all four functions on host tensors."""
    bf, i32 = torch.bfloat16, torch.int32
    x, dx, gain = torch.ones(4, 128, dtype=bf), torch.ones(4, 128, dtype=bf), torch.ones(64)
    fr = torch.zeros(32, dtype=torch.float64)
    kp, gp = tg.cache_pools(4, 16, 2, 64, 104, device="cpu")
    batch = (torch.zeros(1, 2, dtype=i32), torch.tensor([0, 4], dtype=i32), torch.tensor([4], dtype=i32))
    g = torch.ones(4, 208, dtype=bf)
    return [lambda: tg.tango_qk_norm_rope(x, None, dx, None, fr, H=2),
            lambda: tg.tango_qk_norm_rope_backward(x, None, dx, None, dx, None, fr, H=2, q_gain=gain, dq_gain=gain.clone()),
            lambda: tg.tango_cache_append(x, x, g, dx, kp, gp, *batch, fr, H=2),
            lambda: tg.tango_paged_aggregate(x, g, torch.ones(4, 208, dtype=bf), kp, gp, *batch, H=2, max_new=4, max_len=4)]


class _NoCalls:
    """The library with its launching functions replaced: a call that gets there is recorded."""

    def __init__(self):
        self.raw, self.calls = tg.load(), []

    def __getattr__(self, name):
        if not name.startswith("tango_"):
            return getattr(self.raw, name)
        return lambda *a: self.calls.append(name) or tg.TG_OK


def test_host_tensors_are_refused_before_the_library_sees_them(lib, monkeypatch):
    fake = _NoCalls()
    monkeypatch.setattr(tg, "_lib", fake)
    for call in _cpu_calls():
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    assert fake.calls == []


def test_calls_run_on_their_tensors_device(lib, monkeypatch):
    """Where another device is current, the tensors' own is made current for the workspace's
    size, the stream and the launch, and given back."""
    seen = []

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            seen.append(self.dev)

        def __exit__(self, *a):
            seen.append("left")
    monkeypatch.setattr(tg, "_current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device", Device)
    with tg._on_device(1):
        assert seen == []
    with tg._on_device(0):
        assert seen == [0]
    assert seen == [0, "left"]


def test_given_workspaces_are_checked():
    """Scratch of another device, or with gaps, is refused."""
    ws = torch.zeros(512, dtype=torch.uint8)
    assert tg._given_ws(ws, -1) is ws
    with pytest.raises(ValueError):
        tg._given_ws(ws, 0)
    with pytest.raises(ValueError):
        tg._given_ws(ws[::2], -1)


def _wide(B, N, max_len, dtype, **kw):
    """A batch at the paper's gate width over pages of 64 tokens."""
    base = dict(B=B, N=N, max_new=-(-N // B), max_len=max_len, m=28480, page_size=64, n_pages=1 << 14,
                table_pitch=-(-max_len // 64), dtype=dtype)
    base.update(kw)
    return _paged(**base)


@pytest.mark.parametrize("B,N,max_len", [(1, 2048, 8192), (1, 8192, 8192), (8, 16384, 8192), (1, 2048, 131072),
                                         (8, 16384, 65536), (257, 768, 32768), (4096, 4096, 131072)])
def test_cuda_core_scratch_stays_within_a_pass(lib, B, N, max_len):
    """Whatever the rows and the length, the weights and partial sums of one pass: 1 GB."""
    for p in (_wide(B, N, max_len, tg.TG_F32), _wide(B, N, max_len, tg.TG_BF16, d_h=128),
              _wide(B, N, max_len, tg.TG_F32, m=9494, max_new=N)):
        assert 0 < tg.tg_workspace_size(tg.TG_WS_PAGED, p) <= (1 << 30) + (1 << 16)


def test_cuda_core_scratch_of_one_tile(lib):
    """Where one tile of 8 rows of one head is more, it is that: 32 bytes a key, and 8 sums of 4
    bytes for every 512 keys and gate (gates in whole blocks of 512 columns)."""
    length = 1 << 22
    p = _wide(1, 64, length, tg.TG_F32)
    most = 32 * length + 8 * 4 * (length // 512) * (28 * 512) + length
    assert (1 << 30) < tg.tg_workspace_size(tg.TG_WS_PAGED, p) <= most


@pytest.mark.parametrize("B,N,max_len", [(8, 65536, 131072), (1, 16384, 262144), (4096, 4096, 262144), (1, 2048, 1 << 20)])
def test_tensor_core_scratch_stays_within_a_pass(lib, B, N, max_len):
    """The weights of one pass within 2 GB (and what goes with them: denominators, partial sums,
    counters: 1/4 GB), where the rows of one head alone would take more."""
    assert 2 * (N + 8 * B) * max_len > 2 << 30
    p = _wide(B, N, max_len, tg.TG_BF16)
    assert 0 < tg.tg_workspace_size(tg.TG_WS_PAGED, p) <= (2 << 30) + (1 << 28)


@pytest.mark.parametrize("B,N,max_len", [(1, 2048, 8192), (8, 16384, 8192), (1, 2048, 131072), (257, 768, 32768),
                                         (32, 32, 8192)])
def test_tensor_core_calls_need_not_bring_the_other_paths_scratch(lib, B, N, max_len):
    """bf16 calls have to hold either path's scratch (an address off 16 bytes takes the CUDA
    cores): that path makes do with the tensor cores' own (weights of 2 bytes a row, key and
    head, and up to 1/4 GB of sums), or 1/4 GB."""
    weights = 2 * 2 * (N + 8 * B + 8) * max_len
    assert 0 < tg.tg_workspace_size(tg.TG_WS_PAGED, _wide(B, N, max_len, tg.TG_BF16)) <= weights + (1 << 28)


def test_lengths_past_the_cuda_core_grids(lib):
    """65,535 spans of 128 keys is what those kernels' grids hold: a longer bound is refused
    with its reason before the workspace is looked at, also where only an address off 16 bytes
    keeps the call from the tensor cores; aligned bf16 calls take it."""
    raw, st = tg.load().tango_paged_aggregate, lambda p, q=A: raw(ctypes.byref(p), q, A, A, A, A, None, 0, None)
    for kw in (dict(dtype=tg.TG_F32), dict(dtype=tg.TG_BF16, d_h=128)):
        kw.update(B=1, N=1, max_new=1, m=128, page_size=1 << 16, table_pitch=1 << 10)
        assert st(_paged(max_len=65535 * 128, **kw)) == tg.TG_ERR_WORKSPACE
        p = _paged(max_len=65535 * 128 + 1, **kw)
        assert st(p) == tg.TG_ERR_UNSUPPORTED and tg.tg_workspace_size(tg.TG_WS_PAGED, p) == 0
    kw.update(d_h=64)
    p = _paged(max_len=65535 * 128 + 1, **kw)
    assert st(p) == tg.TG_ERR_WORKSPACE and st(p, A + 2) == tg.TG_ERR_UNSUPPORTED
    assert tg.tg_workspace_size(tg.TG_WS_PAGED, p) > 0


def test_paged_flags(lib):
    """The test hook is the only flag of these parameters."""
    raw, P = tg.load(), ctypes.byref
    for flags, status in ((tg.TG_FLAG_DEBUG_TIMEOUT, tg.TG_ERR_WORKSPACE), (tg.TG_FLAG_QK_NORMALIZED, tg.TG_ERR_INVALID_ARG),
                          (1 << 31, tg.TG_ERR_INVALID_ARG)):
        assert raw.tango_paged_aggregate(P(_paged(flags=flags)), A, A, A, A, A, None, 0, None) == status
    assert raw.tango_cache_append(P(_paged(flags=2)), P(_append()), A, A, A, A, A, A, None) == tg.TG_ERR_INVALID_ARG
    assert tg.tg_workspace_size(tg.TG_WS_PAGED, _paged(flags=2)) == 0
