"""The float64 forms the 8-bit operators and the norms are tested against (plain64.py), against
exact rationals, integer products, torch's own norms in float64 and the C oracle; and their error
bounds against an fp32 evaluation of the same formulas (CPU only)."""
from fractions import Fraction

import numpy as np
import pytest
import torch
import torch.nn.functional as F

import oracle
import plain64


def _round_half_even(f):
    n = f.numerator // f.denominator
    r = f - n
    return n + (1 if r > Fraction(1, 2) or (r == Fraction(1, 2) and n % 2) else 0)


def test_codes_are_the_rationals_rounded():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(20, 64, generator=g).to(torch.bfloat16).double().numpy()
    x[0, 0], x[0, 1] = x[0].max() * 2, x[0].max()          # a tie: half the largest is 63.5
    x[1] = np.sign(x[1]) * np.arange(64) / 2               # 254 / 8 = 31.75 at the end: no ties
    x[2] = np.arange(64) * 2.0 - 63                        # odd numbers
    x[2, 0] = 127.0                                        # codes are the values
    x[3] = 0
    q, s = plain64.codes(x)
    for r in range(20):
        amax = max(abs(Fraction(float(v))) for v in x[r])
        want = [_round_half_even(Fraction(float(v)) * 127 / amax) if amax else 0 for v in x[r]]
        assert q[r].tolist() == want
        assert abs(Fraction(float(s[r])) - amax / 127) <= amax / 127 * Fraction(1, 2 ** 52)
    bad = np.array([[1.0, np.nan], [np.inf, 2.0], [-np.inf, np.nan], [3.0, -1.5]])
    q, s = plain64.codes(bad)
    assert (q[:3] == 0).all() and np.isnan(s[:3]).all() and q[3].tolist() == [127, -64]


def test_check_codes_catches_a_wrong_code():
    v = np.random.default_rng(0).normal(size=(4, 40))
    q, s = plain64.codes(v)
    tol = np.zeros_like(v)
    plain64.check_codes(q, s, v, tol)
    for wrong in (q + 1 * (np.arange(40) == 7), np.roll(q, 1, 1)):
        with pytest.raises(AssertionError):
            plain64.check_codes(np.clip(wrong, -127, 127), s, v, tol)
    with pytest.raises(AssertionError):
        plain64.check_codes(q, s * (1 + 1e-5), v, tol)


def test_linear_against_integer_products():
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-127, 128, (6, 90), generator=g)
    w = torch.randint(-127, 128, (8, 90), generator=g)
    xs, ws = torch.rand(6, generator=g).double(), torch.rand(8, generator=g).double()
    b, a = torch.randn(8, generator=g).double(), torch.randn(6, 8, generator=g).double()
    ref, tol = plain64.linear(x, xs, w, ws, b, a)
    want = (x @ w.T).double() * xs[:, None] * ws + b + a
    assert np.allclose(ref, want.numpy(), rtol=1e-14, atol=0)
    f32 = ((x @ w.T).float() * xs.float()[:, None]) * ws.float() + b.float() + a.float()
    inputs = 3 * plain64.U * np.abs((x @ w.T).numpy() * xs.numpy()[:, None] * ws.numpy())  # xs, ws in fp32
    assert (np.abs(f32.double().numpy() - ref) <= tol + inputs + plain64.U * (b.abs() + a.abs()).numpy()).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norms_against_torch(kind):
    g = torch.Generator().manual_seed(2)
    v = (torch.randn(3, 5, 72, generator=g) * 3 + 1).double()
    f = (lambda t: F.rms_norm(t, (72,), eps=1e-3)) if kind == "rms" else (lambda t: F.layer_norm(t, (72,), eps=1e-3))
    ref, tol = plain64.norm(v.numpy(), kind, 1e-3)
    assert np.allclose(ref, f(v).numpy(), rtol=1e-12, atol=1e-13)
    assert (np.abs(f(v.float()).double().numpy() - plain64.norm(v.float().double().numpy(), kind, 1e-3)[0]) <= tol).all()


def test_block_norm_against_torch():
    g = torch.Generator().manual_seed(3)
    B, n, C = 3, 4, 40
    x, y = torch.randn(B, n, C, generator=g).double(), torch.randn(B, n, C, generator=g).double()
    wo, wi = torch.rand(C, generator=g).double() + 0.5, torch.rand(C, generator=g).double() + 0.5
    gate, scale, shift = (torch.randn(B, C, generator=g).double() for _ in range(3))
    (r, dr), (h, dh) = plain64.block_norm(x, y, wo, gate, 0.75, "layer", wi, scale, shift, "rms", 1e-4)
    want_r = 0.75 * x + gate[:, None] * F.layer_norm(y, (C,), wo, eps=1e-4)
    want_h = F.rms_norm(want_r, (C,), wi, eps=1e-4) * (1 + scale[:, None]) + shift[:, None]
    assert np.allclose(r, want_r.numpy(), rtol=1e-12, atol=1e-13) and np.allclose(h, want_h.numpy(), rtol=1e-11, atol=1e-12)
    assert (dr > 0).all() and (dh > 0).all() and dh.max() < 1e-3
    none, (h, _) = plain64.block_norm(x, pre="layer")
    assert none is None and np.allclose(h, F.layer_norm(x, (C,), eps=1e-6).numpy(), rtol=1e-11, atol=1e-12)
    (r, _), _ = plain64.block_norm(x, y, post="none", alpha=-1.0)
    assert np.allclose(r, (y - x).numpy(), rtol=1e-14)


def test_gate_norm_against_the_oracle():
    g = torch.Generator().manual_seed(4)
    y, z, w = torch.randn(7, 96, generator=g), torch.randn(7, 96, generator=g) * 4, torch.rand(96, generator=g)
    ref, _ = plain64.gate_norm(y, z, w, 32, 1e-5)
    assert np.allclose(ref, oracle.get().gate_norm(y.double().numpy(), z.double().numpy(), w.double().numpy(), 32, 1e-5),
                       rtol=1e-12, atol=1e-14)
