"""The norms around a block (mate_block_norm_fwd) against plain float64 (plain64.py, which derives
the bounds), over both norms, storage types and halves, and the shapes and strides of a user's
modulation tensors."""
import numpy as np
import pytest
import torch

import plain64
from gpu_util import host64

pytestmark = pytest.mark.gpu

mate = pytest.importorskip("linear_complexity_video_b200")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mate.load()


def _inputs(B, n, C, seed, x_dtype=torch.bfloat16, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    t = dict(x=(torch.randn(B, n, C, generator=g) * 2 + offset).to(x_dtype),
             y=(torch.randn(B, n, C, generator=g) + offset).to(torch.bfloat16),
             w_post=1 + torch.randn(C, generator=g) / 10, w_pre=1 + torch.randn(C, generator=g) / 10,
             mod=torch.randn(B, 3 * C, generator=g) / 3)
    t["shift"], t["scale"], t["gate"] = t["mod"].split(C, 1)
    return t


def _dev(t):
    d = {k: v.cuda() for k, v in t.items() if k in ("x", "y", "w_post", "w_pre", "mod")}
    C = t["x"].shape[-1]
    d["shift"], d["scale"], d["gate"] = d["mod"].split(C, 1)  # column ranges of one tensor
    return d


def _check(got, ref, tol, dtype):
    half = plain64.HALF_STEP["bf16" if dtype == torch.bfloat16 else "f32"]
    off, limit = np.abs(host64(got) - ref), tol + half * (np.abs(ref) + tol) + 1e-40
    assert (off <= limit).all(), float((off / limit).max())


def _run(t, norm, post, has_y, h_dtype, alpha, eps=1e-6, B=None):
    d = _dev(t)
    after = dict(y=d["y"], w_post=d["w_post"], gate=d["gate"], residual_scale=alpha, post_norm=post) if has_y else {}
    if has_y and not post:
        after["w_post"] = None
    before = dict(w_pre=d["w_pre"], scale=d["scale"], shift=d["shift"]) if h_dtype is not None else {}
    r, h = mate.block_norm(d["x"], **after, **before, norm=norm, eps=eps, h_dtype=h_dtype)
    first, second = plain64.block_norm(t["x"].double(), t["y"].double() if has_y else None,
                                       t["w_post"].double() if post else None, t["gate"].double(), alpha,
                                       norm if post else "none", t["w_pre"].double(), t["scale"].double(),
                                       t["shift"].double(), norm, eps)
    if has_y:
        assert r.dtype == t["x"].dtype and r.shape == t["x"].shape
        _check(r, *first, t["x"].dtype)
    else:
        assert r is None
    if h_dtype == torch.bfloat16:
        _check(h, *second, torch.bfloat16)
    elif h_dtype == torch.int8:
        plain64.check_codes(host64(h.q), host64(h.scale), *second)
    else:
        assert h is None


SHAPES = [(1, 1, 8), (2, 1, 2560), (3, 1155, 64), (1, 13, 1280), (2, 37, 1288), (3, 50, 2560), (1, 21, 2568),
          (2, 9, 5120), (1, 7, 5128), (2, 5, 8192), (5, 3, 40), (700, 1, 72), (1, 2000, 320)]


@pytest.mark.parametrize("h_dtype", [torch.bfloat16, torch.int8], ids=["bf16", "i8"])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("B,n,C", SHAPES)
def test_after_and_before(B, n, C, norm, h_dtype):
    x_dtype = torch.float32 if (B + n + C // 8) % 2 else torch.bfloat16
    _run(_inputs(B, n, C, seed=B + n + C, x_dtype=x_dtype), norm, True, True, h_dtype, 0.875)


@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("post,has_y,h_dtype", [(False, True, torch.bfloat16), (False, True, None), (True, True, None),
                                                (False, False, torch.bfloat16), (False, False, torch.int8)])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_halves(norm, post, has_y, h_dtype, x_dtype):
    for B, n, C in ((2, 33, 2560), (3, 5, 136), (1, 3, 6400)):
        _run(_inputs(B, n, C, seed=n, x_dtype=x_dtype), norm, post, has_y, h_dtype, -1.5 if has_y else 1.0)


def test_defaults_are_neutral_and_vectors_broadcast():
    t = _inputs(3, 11, 264, seed=1)
    d = _dev(t)
    r, h = mate.block_norm(d["x"], d["y"])
    first, second = plain64.block_norm(t["x"].double(), t["y"].double())
    _check(r, *first, torch.bfloat16)
    _check(h, *second, torch.bfloat16)
    # one vector for all batch elements: as (C,), as an expanded view, and repeated
    one = dict(gate=d["gate"][0].contiguous(), scale=d["scale"][0].contiguous(), shift=d["shift"][0].contiguous())
    want = mate.block_norm(d["x"], d["y"], **{k: v.repeat(3, 1) for k, v in one.items()})
    for form in (one, {k: v.expand(3, -1) for k, v in one.items()}):
        got = mate.block_norm(d["x"], d["y"], **form)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # each vector with a stride of its own
    got = mate.block_norm(d["x"], d["y"], gate=d["gate"][:1].expand(3, -1), scale=d["scale"].contiguous(), shift=one["shift"])
    want = mate.block_norm(d["x"], d["y"], gate=one["gate"], scale=d["scale"], shift=one["shift"].repeat(3, 1))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a modulation tensor whose columns start off a 16-byte boundary
    m = torch.randn(3, 3 * 264 + 1, device="cuda")
    a = mate.block_norm(d["x"], scale=m[:, 1:265])
    b = mate.block_norm(d["x"], scale=m[:, 1:265].contiguous())
    assert torch.equal(a[1], b[1])


def test_large_mean_keeps_the_layer_norm():
    """Values whose mean is 2,000 times their spread: the squares are taken about the mean."""
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(1, 20, 2560, generator=g) + 2000).float()
    _, h = mate.block_norm(x.cuda(), norm="layer", eps=0.0)
    ref, tol = plain64.block_norm(x.double(), pre="layer", eps=0.0)[1]
    _check(h, ref, tol, torch.bfloat16)
    assert abs(host64(h).std() - 1) < 0.05


@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_in_place_and_rows_behind(x_dtype):
    t = _inputs(1, 301, 2560, seed=4, x_dtype=x_dtype)
    d = _dev(t)
    want = mate.block_norm(d["x"], d["y"], gate=d["gate"], residual_scale=0.5)
    buf = torch.full((1, 303, 2560), 9.0, dtype=x_dtype, device="cuda")
    x = buf[:, :301]
    x.copy_(d["x"])
    r, h = mate.block_norm(x, d["y"], gate=d["gate"], residual_scale=0.5, x_out=x)
    assert r.data_ptr() == x.data_ptr() and torch.equal(r, want[0]) and torch.equal(h, want[1])
    assert (buf[:, 301:] == 9).all()


def test_zero_and_not_finite_rows():
    x = torch.ones(1, 6, 72)
    x[0, 1] = 0
    x[0, 2, 71] = float("nan")
    x[0, 3, 0] = float("inf")
    x[0, 4] = 1e-30
    for dt in (torch.float32, torch.bfloat16):
        _, h = mate.block_norm(x.to(dt).cuda(), h_dtype=torch.int8)
        q, s = host64(h.q)[0], host64(h.scale)[0]
        assert (q[0] == 127).all() and (q[5] == 127).all()
        assert (q[1] == 0).all() and s[1] == 0
        assert (q[2:4] == 0).all() and np.isnan(s[2:4]).all()
        assert (q[4] == 127).all() and 0 < s[4] < 1e-20  # 1e-30 / sqrt(1e-6) / 127
        _, h = mate.block_norm(x.to(dt).cuda())
        assert torch.isnan(h[0, 2]).all() and (h[0, 1] == 0).all() and torch.isfinite(h[0, [0, 1, 4, 5]]).all()


def test_h_follows_the_unrounded_residual():
    """h comes from r in fp32: with a bf16 stream it is nearer the exact value than a second call
    on the stored r would be."""
    t = _inputs(1, 64, 2560, seed=9)
    d = _dev(t)
    r, h = mate.block_norm(d["x"], d["y"])
    _, again = mate.block_norm(r)
    ref = plain64.block_norm(t["x"].double(), t["y"].double())[1][0]
    one, two = (np.linalg.norm(host64(v) - ref) for v in (h, again))
    assert one < 0.9 * two


def test_stream_argument_and_many_rows():
    t = _inputs(2, 5000, 128, seed=2)
    d = _dev(t)
    want = mate.block_norm(d["x"], d["y"], gate=d["gate"], h_dtype=torch.int8)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = mate.block_norm(d["x"], d["y"], gate=d["gate"], h_dtype=torch.int8, stream=st)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1].q, want[1].q) and torch.equal(got[1].scale, want[1].scale)


@pytest.mark.slow
def test_two_grids_of_73728_tokens():
    B, n, C = 2, 73728, 2560
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(B, n, C, generator=g, device="cuda").to(torch.bfloat16)
    y = torch.randn(B, n, C, generator=g, device="cuda").to(torch.bfloat16)
    gate = torch.randn(B, C, generator=g, device="cuda")
    r, h = mate.block_norm(x, y, gate=gate, h_dtype=torch.int8)
    for b, rows in ((0, [0, 1, 40000, n - 1]), (1, [0, 33333, n - 2, n - 1])):
        first, second = plain64.block_norm(host64(x[b:b + 1, rows]), host64(y[b:b + 1, rows]), gate=host64(gate[b:b + 1]))
        _check(r[b:b + 1, rows], *first, torch.bfloat16)
        plain64.check_codes(host64(h.q[b:b + 1, rows]), host64(h.scale[b:b + 1, rows]), *second)
