"""Sizes past the library's 32-bit integers are refused by the binding, not cut to their low bits (CPU only)."""
import ctypes

import pytest

import linear_complexity_video_b200 as mate
from linear_complexity_video_b200 import _lib, api

DIMS = [c for c in vars(_lib).values() if isinstance(c, type) and issubclass(c, _lib.Dims) and c is not _lib.Dims]


@pytest.mark.parametrize("cls", DIMS, ids=lambda c: c.__name__)
def test_dims_refuse_what_their_fields_cannot_hold(cls):
    ones = {n: 1 for n, _ in cls._fields_}
    values = list(range(3, 3 + len(ones)))
    for d in (cls(*values), cls.of(*values), cls(**dict(zip(ones, values)))):
        assert [getattr(d, n) for n in ones] == values
    assert [getattr(cls(7), n) for n in ones] == [7] + [0] * (len(ones) - 1)
    for i, (n, t) in enumerate(cls._fields_):
        if t is ctypes.c_float:
            continue
        bits = 8 * ctypes.sizeof(t)
        for good in (-2 ** (bits - 1), 2 ** (bits - 1) - 1):
            v = values[:i] + [good] + values[i + 1:]
            assert getattr(cls(*v), n) == getattr(cls.of(*v), n) == good
        for bad in (2 ** (bits - 1), 2 ** bits + 5, -2 ** (bits - 1) - 1):
            v = values[:i] + [bad] + values[i + 1:]
            for make in (lambda: cls(*v), lambda: cls.of(*v), lambda: cls(**{**ones, n: bad})):
                with pytest.raises(ValueError, match="does not fit"):
                    make()


def test_entry_point_integers():
    mate.load()
    d = _lib.mate_ssd_dims(1, 4, 64, 64, 1, 256, 1, 3)
    assert api.mate_bissd_workspace_bytes(8, 16, 16, None, d) > 0
    for grid in ((2 ** 32 + 8, 16, 16), (8, 16 - 2 ** 32, 16), (8, 16, 2 ** 31)):
        with pytest.raises((ValueError, ctypes.ArgumentError), match="does not fit"):
            api.mate_bissd_workspace_bytes(*grid, None, d)
    with pytest.raises(ValueError, match="does not fit"):
        api.mate_bissd_workspace_bytes(8, 16, 16, (2 ** 32 + 4, 4, 4), d)
    assert _lib.Int.from_param(ctypes.c_int(5)).value == 5


@pytest.mark.parametrize("d_model,want", [(131072, _lib.MATE_ERR_INVALID_ARG), (131136, _lib.MATE_ERR_UNSUPPORTED),
                                          (1 << 24, _lib.MATE_ERR_UNSUPPORTED)])
def test_frontend_i8_takes_no_longer_sums_than_the_linear_layer(d_model, want):
    """int32 holds sums of 131,072 products of codes: the front-end's in_proj has that limit too. (The
    call that is in bounds is refused for its null pointers, behind the check of its sizes.)"""
    L, d = mate.load(), _lib.mate_frontend_dims(1, d_model, 8, 64, 1, 64, _lib.MATE_BF16)
    null = ctypes.c_void_p(0)
    got = L.mate_frontend_i8_fwd(*[null] * 7, 4, 8, 8, 0, *[null] * 5, ctypes.byref(d), null, 0, null)
    assert got == want
