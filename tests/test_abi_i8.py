"""Refusals of the 8-bit operators and the norms around a block: every bad argument is found on
the host, before any CUDA call (no GPU needed; the addresses are never read)."""
import ctypes

import pytest
import torch

import linear_complexity_video_b200 as mate
from linear_complexity_video_b200 import _lib

INVALID, UNSUPPORTED = _lib.MATE_ERR_INVALID_ARG, _lib.MATE_ERR_UNSUPPORTED
BF16, F32, I8 = _lib.MATE_BF16, _lib.MATE_F32, _lib.MATE_I8
BASE, GAP = 1 << 44, 1 << 40


def _p(i, off=0):
    return BASE + i * GAP + off


def test_quant_rows_refusals():
    L = mate.load()

    def call(d, x=_p(0), q=_p(1), s=_p(2)):
        return L.mate_quant_rows_fwd(x, q, s, None if d is None else ctypes.byref(_lib.mate_quant_dims(*d)), None)

    ok = (4, 64, BF16)
    assert call(None) == INVALID
    for d in ((0, 64, BF16), (-1, 64, BF16), (4, 0, BF16), (4, -8, BF16)):
        assert call(d) == INVALID, d
    for d in ((4, 64, F32), (4, 60, BF16), (4, 20488, BF16), (4, 64, 7)):
        assert call(d) == UNSUPPORTED, d
    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(x=_p(0, 8)), dict(q=_p(1, 8)), dict(s=_p(2, 2))):
        assert call(ok, **kw) == INVALID, kw
    # overlaps: codes over the input's last bytes, scales over the input or the codes
    assert call(ok, q=_p(0, 4 * 64 * 2 - 16)) == INVALID
    assert call(ok, s=_p(0, 16)) == INVALID
    assert call(ok, s=_p(1, 4 * 64 - 4)) == INVALID


def test_linear_i8_refusals():
    L = mate.load()

    def call(d, **kw):
        a = dict(x=_p(0), xs=_p(1), w=_p(2), ws=_p(3), bias=None, add=None, out=_p(6))
        a.update(kw)
        return L.mate_linear_i8_fwd(a["x"], a["xs"], a["w"], a["ws"], a["bias"], a["add"], a["out"],
                                    None if d is None else ctypes.byref(_lib.mate_linear_i8_dims(*d)), None)

    ok = (128, 256, 64, BF16)
    assert call(None) == INVALID
    for d in ((0, 256, 64, BF16), (128, 0, 64, BF16), (128, 256, 0, BF16), (-5, 256, 64, BF16)):
        assert call(d) == INVALID, d
    for d in ((128, 256, 64, I8), (128, 250, 64, BF16), (128, 8, 64, BF16), (128, 256, 60, BF16),
              (128, 131088, 64, BF16), (128, 256, 64, 9), (2**31 - 1, 256, 64, BF16), (128, 256, 2**31 - 8, BF16)):
        assert call(d) == UNSUPPORTED, d
    for n in ("x", "xs", "w", "ws", "out"):
        assert call(ok, **{n: None}) == INVALID, n
    for n, i in (("x", 0), ("w", 2), ("ws", 3), ("out", 6)):
        assert call(ok, **{n: _p(i, 8)}) == INVALID, n
    assert call(ok, xs=_p(1, 2)) == INVALID
    assert call(ok, bias=_p(4, 4)) == INVALID and call(ok, add=_p(5, 8)) == INVALID
    out_bytes = 128 * 64 * 2
    for n, i in (("x", 0), ("xs", 1), ("w", 2), ("ws", 3)):
        assert call(ok, out=_p(i)) == INVALID, n
    assert call(ok, bias=_p(6)) == INVALID
    assert call(ok, add=_p(6, 16)) == INVALID and call(ok, add=_p(6, out_bytes - 16)) == INVALID


def test_gate_norm_i8_refusals():
    L = mate.load()

    def call(d, eps=1e-5, **kw):
        a = dict(y=_p(0), z=_p(1), w=_p(2), q=_p(3), s=_p(4))
        a.update(kw)
        return L.mate_gate_norm_i8_fwd(a["y"], a["z"], a["w"], ctypes.c_float(eps), a["q"], a["s"],
                                       None if d is None else ctypes.byref(_lib.mate_gate_norm_dims(*d)), None)

    ok = (16, 64, 32, BF16)
    assert call(None) == INVALID
    for d in ((0, 64, 32, BF16), (16, 0, 32, BF16), (16, 64, 0, BF16)):
        assert call(d) == INVALID, d
    for d in ((16, 64, 48, BF16), (16, 60, 12, BF16), (16, 8200, 8200, BF16), (16, 64, 32, F32), (16, 64, 32, I8)):
        assert call(d) == UNSUPPORTED, d
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(ok, eps=eps) == INVALID, eps
    for n in ("y", "z", "w", "q", "s"):
        assert call(ok, **{n: None}) == INVALID, n
    for n, i in (("y", 0), ("z", 1), ("w", 2), ("q", 3)):
        assert call(ok, **{n: _p(i, 8)}) == INVALID, n
    assert call(ok, s=_p(4, 1)) == INVALID
    assert call(ok, q=_p(0, 16)) == INVALID and call(ok, q=_p(1)) == INVALID and call(ok, s=_p(2)) == INVALID
    assert call(ok, s=_p(3, 16 * 64 - 4)) == INVALID


def test_block_norm_refusals():
    L = mate.load()
    names = ("x", "y", "w_post", "gate", "w_pre", "scale", "shift", "x_out", "h", "h_scale")

    def dims(**kw):
        a = dict(batch=2, tokens=8, channels=64, post_norm=1, pre_norm=1, x_dtype=BF16, h_dtype=BF16, gate_stride=192,
                 scale_stride=128, shift_stride=64, residual_scale=1.0, eps=1e-6)
        a.update(kw)
        return _lib.mate_block_norm_dims(*a.values())

    def call(d=dims(), **kw):
        a = {n: _p(i) for i, n in enumerate(names)}
        a["h_scale"] = None
        a.update(kw)
        return L.mate_block_norm_fwd(*a.values(), None if d is None else ctypes.byref(d), None)

    assert call(None) == INVALID
    for kw in (dict(batch=0), dict(tokens=0), dict(channels=0), dict(channels=-8), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(residual_scale=float("nan")),
               dict(residual_scale=float("inf")), dict(gate_stride=-1), dict(scale_stride=-1), dict(shift_stride=-1)):
        assert call(dims(**kw)) == INVALID, kw
    for kw in (dict(channels=60), dict(channels=8200), dict(x_dtype=I8), dict(h_dtype=F32), dict(h_dtype=9),
               dict(post_norm=3), dict(post_norm=-1), dict(pre_norm=0), dict(pre_norm=3),
               dict(batch=1 << 16, tokens=1 << 15), dict(gate_stride=1 << 31), dict(shift_stride=1 << 62)):
        assert call(dims(**kw)) == UNSUPPORTED, kw
    # x is always there; y and x_out come together; something has to be asked for
    assert call(x=None) == INVALID and call(y=None) == INVALID and call(x_out=None) == INVALID
    none = dict(y=None, x_out=None, w_post=None, gate=None)
    assert call(**none, h=None, w_pre=None, scale=None, shift=None) == INVALID
    # vectors of a half that is not asked for
    assert call(y=None, x_out=None, gate=None) == INVALID and call(y=None, x_out=None, w_post=None) == INVALID
    for n in ("w_pre", "scale", "shift"):
        kw = dict(h=None, w_pre=None, scale=None, shift=None)
        kw[n] = _p(5)
        assert call(**kw) == INVALID, n
    # scales exactly with 8-bit codes
    assert call(h_scale=_p(9)) == INVALID and call(dims(h_dtype=I8)) == INVALID
    for n in ("x", "y", "x_out", "h"):
        assert call(**{n: _p(names.index(n), 8)}) == INVALID, n
    for n in ("w_post", "gate", "w_pre", "scale", "shift"):
        assert call(**{n: _p(names.index(n), 2)}) == INVALID, n
    assert call(dims(h_dtype=I8), h_scale=_p(9, 2)) == INVALID
    # overlaps; a modulation vector reaches over (batch - 1) strides of its own
    assert call(x_out=_p(0, 16)) == INVALID and call(x_out=_p(1)) == INVALID and call(h=_p(0)) == INVALID
    assert call(h=_p(7, 2 * 8 * 64 * 2 - 16)) == INVALID
    for n, stride in (("gate", 192), ("scale", 128), ("shift", 64)):
        assert call(h=_p(names.index(n), stride * 4 + 64 * 4 - 16)) == INVALID, n
    assert call(dims(h_dtype=I8), h_scale=_p(0, 64)) == INVALID
    assert call(x_out=_p(0), h=_p(0, 512)) == INVALID  # in place, and h over both


def test_frontend_i8_refusals():
    L = mate.load()
    d = _lib.mate_frontend_dims(1, 256, 8, 64, 1, 64, BF16)
    nbytes = L.mate_frontend_workspace_bytes(4, 8, 8, ctypes.byref(d))
    names = ("u", "us", "w", "ws", "cw", "cb", "db")

    def call(dd=d, mode=0, n=nbytes, **kw):
        a = {k: _p(i) for i, k in enumerate(names)}
        outs = {k: _p(10 + i) for i, k in enumerate(("z", "x", "dt", "B", "C"))}
        a.update({k: v for k, v in kw.items() if k in a})
        outs.update({k: v for k, v in kw.items() if k in outs})
        return L.mate_frontend_i8_fwd(*a.values(), 4, 8, 8, mode, *outs.values(),
                                      None if dd is None else ctypes.byref(dd), kw.get("work", _p(20)),
                                      ctypes.c_size_t(n), None)

    assert call(None) == INVALID and call(mode=5) == INVALID
    assert call(_lib.mate_frontend_dims(1, 100, 8, 64, 1, 64, BF16)) == UNSUPPORTED
    assert call(_lib.mate_frontend_dims(1, 256, 8, 64, 1, 64, F32)) == UNSUPPORTED
    for n in names + ("z", "x", "dt", "B", "C"):
        assert call(**{n: None}) == INVALID, n
    assert call(us=_p(1, 2)) == INVALID and call(ws=_p(3, 8)) == INVALID and call(u=_p(0, 8)) == INVALID
    assert call(n=nbytes - 1) == _lib.MATE_ERR_WORKSPACE and call(work=None) == _lib.MATE_ERR_WORKSPACE
    assert call(z=_p(1)) == INVALID and call(dt=_p(3)) == INVALID and call(x=_p(10)) == INVALID


def test_python_entry_points_refuse_host_tensors():
    b, f, i = torch.bfloat16, torch.float32, torch.int8
    z = lambda *s, dtype=b: torch.zeros(*s, dtype=dtype)  # noqa: E731
    for call in (lambda: mate.quantize_rows(z(4, 64)),
                 lambda: mate.linear_i8(z(4, 64, dtype=i), z(4, dtype=f), z(8, 64, dtype=i), z(8, dtype=f)),
                 lambda: mate.gate_norm_i8(z(4, 64), z(4, 64), z(64, dtype=f), 64),
                 lambda: mate.block_norm(z(1, 4, 64)),
                 lambda: mate.modulation(z(1, 64), mate.Codes(z(192, 64, dtype=i), z(192, dtype=f)))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_block_norm_refuses_arguments_without_their_half():
    x = torch.zeros(1, 4, 64)
    for kw in (dict(gate=x), dict(w_post=x), dict(x_out=x), dict(residual_scale=2.0), dict(h_dtype=None),
               dict(h_dtype=torch.float16), dict(norm="batch")):
        with pytest.raises(ValueError):
            mate.block_norm(x, **kw)
    with pytest.raises(ValueError, match="go with h"):
        mate.block_norm(x, x, h_dtype=None, scale=x)
