"""Host-side checks of lookup, norm, distillation and sampling: bad arguments are refused before
anything is launched, on a machine without a GPU too."""
import ctypes
import math

import pytest
import torch

import cross_token_gated_gb300 as tg

A = 256  # a pointer that validation never follows
BAD, NO, WS = tg.TG_ERR_INVALID_ARG, tg.TG_ERR_UNSUPPORTED, tg.TG_ERR_WORKSPACE


def _embed(**kw):
    base = dict(rows=4, d=64, vocab=100, scale=1.0, pad_id=-1, pitch=0, dtype=tg.TG_BF16, grad_dtype=tg.TG_F32)
    return tg.tg_embed_params(*(base | kw).values())


def _norm(**kw):
    base = dict(rows=4, d=64, norm=tg.TG_NORM_RMS, eps=1e-6, x_pitch=0, dtype=tg.TG_BF16)
    return tg.tg_norm_params(*(base | kw).values())


def _distill(**kw):
    base = dict(rows=4, vocab=100, k=8, temperature=1.0, pitch=0, grad_pitch=0, dtype=tg.TG_BF16)
    return tg.tg_distill_params(*(base | kw).values())


def _sample(**kw):
    base = dict(rows=4, vocab=100, pitch=0, dtype=tg.TG_BF16, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
                temperatures=None, top_ks=None, top_ps=None, min_ps=None)
    return tg.tg_sample_params(*(base | kw).values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(d=0), BAD), (dict(vocab=0), BAD), (dict(dtype=2), BAD), (dict(grad_dtype=-1), BAD),
    (dict(pitch=63), BAD), (dict(rows=(1 << 30) + 1), NO), (dict(vocab=(1 << 28) + 1), NO), (dict(d=(1 << 24) + 1), NO),
])
def test_embed_refusals(lib, kw, status):
    raw, p = tg.load(), _embed(**kw)
    assert raw.tango_embed(ctypes.byref(p), A, A, A, None) == status
    assert raw.tango_embed_backward(ctypes.byref(p), A, A, None, A, A, 1 << 40, None) == status
    assert tg.tg_workspace_size(tg.TG_WS_EMBED_BWD, p) == 0


def test_embed_pointer_refusals(lib):
    raw, p = tg.load(), _embed()
    f, b, ref = raw.tango_embed, raw.tango_embed_backward, ctypes.byref(_embed())
    need = tg.tg_workspace_size(tg.TG_WS_EMBED_BWD, p)
    assert need > 0 and need % 256 == 0
    for bad in ((None, A, A, A), (ref, None, A, A), (ref, A, None, A), (ref, A, A, None)):
        assert f(*bad, None) == BAD
    assert f(ref, A + 2, A, A, None) == NO and f(ref, A, A + 1, A, None) == NO
    assert b(ref, A, None, None, A, A, need, None) == BAD
    assert b(ref, A, A, None, None, A, need, None) == BAD
    assert b(ref, A, A, None, A + 2, A, need, None) == NO            # a float gradient
    assert b(ref, A, A, None, A, None, 0, None) == WS
    assert b(ref, A, A, None, A, A, need - 1, None) == WS
    assert b(ref, A, A, None, A, A + 16, need, None) == WS
    assert f(ctypes.byref(_embed(rows=0)), None, A, None, None) == tg.TG_OK


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(d=0), BAD), (dict(norm=tg.TG_NORM_NONE), BAD), (dict(norm=tg.TG_NORM_UNIT), BAD),
    (dict(norm=4), BAD), (dict(eps=0.0), BAD), (dict(eps=math.nan), BAD), (dict(x_pitch=63), BAD), (dict(dtype=2), BAD),
    (dict(d=(1 << 24) + 1), NO),
])
def test_norm_refusals(lib, kw, status):
    raw, p = tg.load(), _norm(**kw)
    assert raw.tango_norm(ctypes.byref(p), A, A, A, A, None) == status
    assert raw.tango_norm_backward(ctypes.byref(p), A, A, A, None, A, A, None, A, 1 << 40, None) == status
    assert tg.tg_workspace_size(tg.TG_WS_NORM_BWD, p) == 0


def test_norm_pointer_refusals(lib):
    raw, p = tg.load(), _norm()
    f, b, ref = raw.tango_norm, raw.tango_norm_backward, ctypes.byref(_norm())
    need = tg.tg_workspace_size(tg.TG_WS_NORM_BWD, p)
    assert f(None, A, A, A, A, None) == BAD and f(ref, None, A, A, A, None) == BAD and f(ref, A, A, A, None, None) == BAD
    assert f(ref, A, A + 1, A, A, None) == NO
    assert b(ref, A, None, A, None, A, A, None, A, need, None) == BAD     # dgamma without gamma
    assert b(ref, A, A, None, None, A, None, None, None, 0, None) == BAD
    assert b(ref, A, A, A, None, A, A, None, None, 0, None) == WS
    assert b(ref, A, A, A, None, A, None, A, A, need - 1, None) == WS
    assert b(ref, A, A, A, None, A, None, A + 2, A, need, None) == NO
    assert f(ctypes.byref(_norm(rows=0)), None, None, None, None, None) == tg.TG_OK
    # the other calls take no layer norm
    q = tg.tg_qk_params(4, 2, 2, 64, 0, 0, tg.TG_NORM_LAYER, 1e-6, 4, None, None, None, None, 0, 0, tg.TG_BF16)
    assert raw.tango_qk_norm_rope(ctypes.byref(q), A, A, A, A, None) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(vocab=0), BAD), (dict(k=0), BAD), (dict(temperature=0.0), BAD),
    (dict(temperature=math.nan), BAD), (dict(temperature=math.inf), BAD), (dict(temperature=-1.0), BAD),
    (dict(pitch=99), BAD), (dict(grad_pitch=99), BAD), (dict(dtype=2), BAD), (dict(k=tg.TG_MAX_TEACHER + 1), NO),
    (dict(vocab=(1 << 24) + 1), NO),
])
def test_distill_refusals(lib, kw, status):
    raw, p = tg.load(), _distill(**kw)
    assert raw.tango_distill(ctypes.byref(p), A, A, A, A, None, None) == status
    assert raw.tango_distill_backward(ctypes.byref(p), A, A, A, A, None, 2 * A, None, None) == status


def test_distill_pointer_refusals(lib):
    raw, ref = tg.load(), ctypes.byref(_distill())
    f, b = raw.tango_distill, raw.tango_distill_backward
    for i in range(4):
        args = [A] * 4
        args[i] = None
        assert f(ref, *args, None, None) == BAD
    assert f(ref, A, A, A, A, A + 4, None) == NO                         # stats come in pairs
    assert b(ref, A, A, A, None, None, A, None, None) == BAD
    assert b(ref, A, A, A, A, A, A, A, None) == BAD                      # loss goes without stats
    assert b(ref, A + 1, A, A, A, None, A, None, None) == NO
    assert b(ctypes.byref(_distill(grad_pitch=128)), A, A, A, A, None, A, None, None) == BAD  # in place: one pitch
    assert f(ctypes.byref(_distill(rows=0)), None, None, None, None, None, None) == tg.TG_OK


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(vocab=0), BAD), (dict(pitch=99), BAD), (dict(dtype=2), BAD),
    (dict(temperature=-0.5), BAD), (dict(temperature=math.nan), BAD), (dict(top_p=math.nan), BAD),
    (dict(min_p=1.5), BAD), (dict(min_p=math.nan), BAD), (dict(vocab=(1 << 19) + 1), NO),
])
def test_sample_refusals(lib, kw, status):
    assert tg.load().tango_sample(ctypes.byref(_sample(**kw)), A, A, A, None, None) == status


def test_sample_refuses_an_infinite_temperature(lib):
    f = tg.load().tango_sample
    assert f(ctypes.byref(_sample(temperature=math.inf)), A, A, A, None, None) == BAD
    assert f(ctypes.byref(_sample(temperature=1e39)), A, A, A, None, None) == BAD  # inf as a float
    assert f(ctypes.byref(_sample(temperature=math.inf, rows=0)), A, A, A, None, None) == BAD
    # the settings of the rows count, and are looked at on the device
    assert f(ctypes.byref(_sample(temperature=math.inf, temperatures=A, rows=0)), A, A, A, None, None) == tg.TG_OK


def test_sample_pointer_refusals(lib):
    f, ref = tg.load().tango_sample, ctypes.byref(_sample())
    assert f(None, A, A, A, None, None) == BAD
    for i in range(3):
        args = [A] * 3
        args[i] = None
        assert f(ref, *args, None, None) == BAD
    assert f(ref, A + 1, A, A, None, None) == NO and f(ref, A, A + 2, A, None, None) == NO
    assert f(ctypes.byref(_sample(top_ks=A + 2)), A, A, A, None, None) == NO
    assert f(ctypes.byref(_sample(rows=0)), None, None, None, None, None) == tg.TG_OK


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_wrong_tensors(lib):
    """Types, shapes and strides are checked before the library is called; host tensors are refused."""
    i32, f32 = torch.int32, torch.float32
    ids, E = _t(4, dtype=i32), _t(10, 8)
    with pytest.raises(ValueError):
        tg.tango_embed(ids, E, _t(4, 8))                                  # a host tensor
    with pytest.raises(TypeError):
        tg.tango_embed(ids.long(), E, _t(4, 8))
    with pytest.raises(ValueError):
        tg.tango_embed(ids, E, _t(3, 8))
    with pytest.raises(ValueError):
        tg.tango_embed(ids, E, _t(4, 7))
    with pytest.raises(ValueError):
        tg.tango_embed(ids, E.t(), _t(4, 10))
    with pytest.raises(ValueError):
        tg.tango_embed_backward(ids, _t(4, 8), _t(10, 8, dtype=f32), base=_t(9, 8, dtype=f32))
    with pytest.raises(TypeError):
        tg.tango_embed_backward(ids, _t(4, 8), _t(10, 8, dtype=torch.float16))
    x = _t(4, 8)
    with pytest.raises(TypeError):
        tg.tango_norm(x, _t(8, dtype=f32), None, x)
    with pytest.raises(ValueError):
        tg.tango_norm(x, _t(7), None, x)
    with pytest.raises(ValueError):
        tg.tango_norm(x, None, None, _t(8, 4).t())
    with pytest.raises(ValueError):
        tg.tango_norm_backward(x, None, _t(3, 8), x)
    z, tl, ti, row = _t(4, 30), _t(4, 3, dtype=f32), _t(4, 3, dtype=i32), _t(4, dtype=f32)
    with pytest.raises(TypeError):
        tg.tango_distill(z, tl.bfloat16(), ti, row)
    with pytest.raises(ValueError):
        tg.tango_distill(z, tl, ti[:, :2], row)
    with pytest.raises(ValueError):
        tg.tango_distill(z, tl, ti, row[:3])
    with pytest.raises(ValueError):
        tg.tango_distill(z, tl, ti, row, stats=row)
    with pytest.raises(ValueError):
        tg.tango_distill_backward(z, tl, ti, row, _t(4, 31))
    tok = _t(4, dtype=i32)
    with pytest.raises(TypeError):
        tg.tango_sample(z, row, tok.long())
    with pytest.raises(TypeError):
        tg.tango_sample(z, row, tok, top_k=row)
    with pytest.raises(ValueError):
        tg.tango_sample(z, row, tok, temperature=row[:2])
    with pytest.raises(ValueError):
        tg.tango_sample(z, row, tok)                                      # a host tensor


def _shape(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")  # has a size, but no memory


def test_binding_refuses_numbers_past_32_bits(lib):
    """The library's int fields would take their low bits: a row of 2^32 + 8 values would be normed as one
    of 8, a padding id of 2^32 + 3 would drop token 3."""
    i32, f32, wide, far = torch.int32, torch.float32, 2 ** 32 + 8, "2\\^31"
    x = _shape(1, wide)
    with pytest.raises(ValueError, match=far):
        tg.tango_norm(x, None, None, x)
    with pytest.raises(ValueError, match=far):
        tg.tango_norm_backward(x, None, x, x)
    with pytest.raises(ValueError, match=far):
        tg.tango_embed(_shape(1, dtype=i32), _shape(wide, 8), _shape(1, 8))
    with pytest.raises(ValueError, match=far):
        tg.tango_embed_backward(_shape(1, dtype=i32), _shape(1, 8), _shape(wide, 8))
    for pad_id in (2 ** 32 + 3, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="pad_id"):
            tg.tango_embed(_t(4, dtype=i32), _t(10, 8), _t(4, 8), pad_id=pad_id)
        with pytest.raises(ValueError, match="pad_id"):
            tg.tango_embed_backward(_t(4, dtype=i32), _t(4, 8), _t(10, 8, dtype=f32), pad_id=pad_id)
    for pad_id in (2 ** 31 - 1, -2 ** 31):
        with pytest.raises(ValueError, match="cpu|host|device"):
            tg.tango_embed(_t(4, dtype=i32), _t(10, 8), _t(4, 8), pad_id=pad_id)
    row = _shape(1, dtype=f32)
    with pytest.raises(ValueError, match=far):
        tg.tango_distill(x, _shape(1, 3, dtype=f32), _shape(1, 3, dtype=i32), row)
    with pytest.raises(ValueError, match=far):
        tg.tango_distill(_shape(1, 30), _shape(1, wide, dtype=f32), _shape(1, wide, dtype=i32), row)
    with pytest.raises(ValueError, match=far):
        tg.tango_sample(x, row, _shape(1, dtype=i32))
    with pytest.raises(ValueError, match=far):
        tg.tango_sample(_shape(wide, 2), _shape(wide, dtype=f32), _shape(wide, dtype=i32))
