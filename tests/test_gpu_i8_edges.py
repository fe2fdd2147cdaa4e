"""The 8-bit operators at their edges: calls that follow one another without a wait, codes and sizes
at the limits, gates far from zero."""
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


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _product(M, K, N, seed):
    g = _gen(seed)
    codes = lambda *s: torch.randint(-127, 128, s, generator=g, dtype=torch.int8, device="cuda")  # noqa: E731
    return (codes(M, K), torch.rand(M, generator=g, device="cuda") + 0.01, codes(N, K),
            torch.rand(N, generator=g, device="cuda") + 0.01)


# Products of the CTA pairs' kernel, where the commits of one CTA arrive at both: one K step (the last
# commits are on their way when the tile's epilogue starts), as many as the ring has stages, one more, and
# many; a single tile column whose second half is empty, and several; pairs with one tile and with several.
PAIRS = [(19200, 128, 128), (19200, 640, 64), (9001, 768, 520), (40000, 16, 264), (6401, 1296, 1000)]
# Those of the few-token kernel: one K step, fewer than its ring's stages, as many, many; one, two and
# four CTAs to a tile; tiles of 16, 32 and 64 tokens.
FEW = [(3, 128, 136), (16, 256, 2560), (30, 768, 18944), (64, 2560, 2560), (300, 1296, 1000)]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("shapes", [PAIRS, FEW], ids=["pairs", "few"])
def test_products_on_the_heels_of_one_another(shapes, captured):
    """A CTA leaves its SM only when nothing more arrives in its shared memory: the next product's CTAs
    have their barriers at the same places. Sixty products without a wait, eager or in one graph,
    against each after a wait."""
    ins = [_product(*s, seed=i) for i, s in enumerate(shapes)]
    want = []
    for a in ins:
        want.append(mate.linear_i8(*a, out_dtype=torch.float32))
        torch.cuda.synchronize()
    for (xq, xs, wq, ws), w in zip(ins, want):
        rows = sorted({min(r, w.shape[0] - 1) for r in (0, 127, 128, 255, 256, w.shape[0])})
        ref, tol = plain64.linear(*(t.cpu() for t in (xq[rows], xs[rows], wq, ws)))
        assert (np.abs(host64(w[rows]) - ref) <= tol + plain64.U * (np.abs(ref) + tol)).all()
    outs = [torch.empty_like(w) for w in want for _ in range(12)]

    def run():
        for i, out in enumerate(outs):
            k = i % len(ins)
            mate.linear_i8(*ins[k], out_dtype=torch.float32, out=outs[12 * k + i // len(ins)])

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        run = graph.replay
    for _ in range(5):
        for out in outs:
            out.fill_(-1.0)
        run()
        torch.cuda.synchronize()
        assert mate.mate_last_error() == 0
        assert all(torch.equal(out, want[i // 12]) for i, out in enumerate(outs))


def test_sizes_past_32_bits_are_refused():
    """2^32 + 8 rows or channels, which would read as 8. The tensors are never read."""
    e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    n = 2 ** 32 + 64
    wide, codes, w = e(1, n), e(1, n, dtype=torch.int8), e(n, dtype=torch.float32)
    one = e(1, dtype=torch.float32)
    for call in (lambda: mate.quantize_rows(wide), lambda: mate.gate_norm_i8(wide, wide, w, n),
                 lambda: mate.block_norm(wide, w_pre=w), lambda: mate.linear_i8(codes, one, e(8, n, dtype=torch.int8), w[:8]),
                 lambda: mate.gate_norm(wide, wide, w, n), lambda: mate.linear(wide, wide)):
        with pytest.raises(ValueError, match="does not fit"):
            call()
    del wide, codes, w
    long = e(2 ** 32 + 8, 8)
    for call in (lambda: mate.quantize_rows(long), lambda: mate.block_norm(long.view(1, -1, 8), h_dtype=torch.int8),
                 lambda: mate.block_norm(long)):
        with pytest.raises(ValueError, match="does not fit"):
            call()
    del long
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(3, 16, 131072), (3, 16, 131056), (1088, 2304, 131072)])
def test_codes_of_minus_128(M, N, K, dtype):
    """The codes that quantise_rows never writes, -128, are exact too: 128 * 128 * 131,072 is 2^31. Rows of
    both kernels (the last shape is the pairs'): all -128; one code off; all 127 against it."""
    x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    x[1, K - 1], x[2], w[5] = -127, 127, 127
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    got = mate.linear_i8(x, one(M), w, one(N), out_dtype=dtype).cpu()
    want = torch.full((M, N), 128.0 * 128 * K, dtype=torch.float64)
    want[1] -= 128
    want[2] = -128.0 * 127 * K
    want[:, 5] = -128.0 * 127 * K
    want[1, 5] += 127
    want[2, 5] = 127.0 * 127 * K
    assert torch.equal(got, want.float().to(dtype))


def _gated_bound(y, z):
    """y SiLU(z) in float64 and how far the kernel's may be from it, u = 2^-24. -z log2 e is off by 2 u of
    itself (its constant and its product), so 2^that by 2 u |z|, and by 4 u more for the approximation (2
    steps); the sum's rounding, the reciprocal (one step, 2 u) and the two products add 5 u:
    9 u + 2 u |z|. The reciprocal of d > 2^126 is flushed to zero, and with it at most |y z| 2^-126."""
    y, z = y.double().numpy(), z.double().numpy()
    with np.errstate(over="ignore"):
        v = y * (z / (1 + np.exp(-z)))
    return v, np.abs(v) * plain64.U * (9 + 2 * np.abs(z)) + np.abs(y * z) * 2.0 ** -126


@pytest.mark.parametrize("M,C,group,spread", [(40, 256, 256, 10), (40, 1032, 344, 30), (33, 5120, 2560, 100),
                                              (25, 64, 16, 1000)])
def test_gate_norm_i8_gates_far_from_zero(M, C, group, spread):
    """Gates of either sign up to several times `spread`: SiLU from 0 (with 2^(-z log2 e) infinite below -88)
    to z itself."""
    g = torch.Generator().manual_seed(C)
    y = torch.randn(M, C, generator=g).to(torch.bfloat16)
    z = (torch.randn(M, C, generator=g) * spread).to(torch.bfloat16)
    z[:, ::7] = torch.linspace(-95, -80, z[:, ::7].numel()).to(torch.bfloat16).view(z[:, ::7].shape)
    w = 1 + torch.randn(C, generator=g) / 10
    got = mate.gate_norm_i8(y.cuda(), z.cuda(), w.cuda(), group, 1e-5)
    v, dv = (t.reshape(M, C // group, group) for t in _gated_bound(y, z))
    N, dN = (t.reshape(M, C) for t in plain64.norm(v, "rms", 1e-5, dv))
    w = w.double().numpy()
    plain64.check_codes(host64(got.q), host64(got.scale), N * w, np.abs(w) * dN + 3 * plain64.U * np.abs(N * w))


def test_gate_norm_i8_large_values_behind_closed_gates():
    """|y z| past fp32's largest where SiLU(z) is 0: the value is 0, as in the bf16 kernel, and the row's
    other values stand. Infinite gates: SiLU(inf) = inf and SiLU(-inf) = -inf * 0, not a number."""
    inf = float("inf")
    y, z = (torch.ones(6, 64, dtype=torch.bfloat16) for _ in range(2))
    y[0, 3], z[0, 3] = 1e20, -1e20
    y[1, 60], z[1, 60] = -3e38, -200.0
    y[2, ::2], z[2, ::2] = 1e30, -1e10
    z[3, 5] = inf
    z[4, 5] = -inf
    for group in (64, 32):
        got = mate.gate_norm_i8(y.cuda(), z.cuda(), torch.ones(64).cuda(), group)
        plain = mate.gate_norm(y.cuda(), z.cuda(), torch.ones(64).cuda(), group)
        q, s, p = host64(got.q), host64(got.scale), host64(plain)
        # each value is 0 or SiLU(1), over the rms of its group (no code is near a border)
        v = np.where((y == 1).numpy(), 1 / (1 + np.exp(-1.0)), 0.0)[[0, 1, 2, 5]]
        N = plain64.norm(v.reshape(4, -1, group), "rms", 1e-5)[0].reshape(4, 64)
        want, scale = plain64.codes(N)
        fine = [0, 1, 2, 5]
        assert np.array_equal(q[fine], want)
        assert (np.abs(s[fine] - scale) <= 2.0 ** -18 * scale).all()
        assert (np.abs(p[fine] - N) <= (2.0 ** -8 + 2.0 ** -18) * N).all()
        assert np.isnan(s[3:5]).all() and (q[3:5] == 0).all()
        assert np.isnan(p[3:5]).any(1).all()


def test_linear_i8_refusals_on_the_device_by_their_code():
    """Calls that only the C entry refuses, each otherwise in order, by the code it gives; and what they
    would have written is as it was."""
    g = _gen(0)
    x = torch.randint(-127, 128, (8, 64), generator=g, dtype=torch.int8, device="cuda")
    w = torch.randint(-127, 128, (8, 64), generator=g, dtype=torch.int8, device="cuda")
    xs, ws = torch.ones(8, device="cuda"), torch.ones(8, device="cuda")
    out = torch.full((8, 8), 3.0, dtype=torch.bfloat16, device="cuda")
    assert mate.linear_i8(x, xs, w, ws, out=out) is out
    out.fill_(3.0)
    over = lambda t: t.view(torch.bfloat16).flatten()[:64].view(8, 8)  # noqa: E731  (the first 128 bytes of t)
    off = torch.zeros(8 * 64 + 8, dtype=torch.int8, device="cuda")[8:].view(8, 64)
    keep = [t.clone() for t in (x, w, out)]
    for args, kw, code in (((x, xs, w, ws), dict(out=over(x)), "INVALID_ARG"),
                           ((x, xs, w, ws), dict(out=over(w)), "INVALID_ARG"),
                           ((x, xs, w, ws), dict(out=out, addend=torch.ones(9, 8, dtype=torch.bfloat16, device="cuda")[1:]), None),
                           ((off, xs, w, ws), dict(out=out), "INVALID_ARG"),
                           ((x, xs, off, ws), dict(out=out), "INVALID_ARG"),
                           ((x[:0], xs[:0], w, ws), {}, "INVALID_ARG"),
                           ((x, xs, w[:0], ws[:0]), {}, "INVALID_ARG"),
                           ((x[:, :0].contiguous(), xs, w[:, :0].contiguous(), ws), dict(out=out), "INVALID_ARG"),
                           ((x[:, :24].contiguous(), xs, w[:, :24].contiguous(), ws), dict(out=out), "UNSUPPORTED"),
                           ((x, xs, w[:4], ws[:4]), {}, "UNSUPPORTED")):
        if code is None:  # the rows of a wider tensor start on their 16 bytes: taken
            mate.linear_i8(*args, **kw)
            out.fill_(3.0)
            continue
        with pytest.raises(mate.MateError) as e:
            mate.linear_i8(*args, **kw)
        assert e.value.code == getattr(mate._lib, "MATE_ERR_" + code)
    with pytest.raises(ValueError, match="must have shape"):
        mate.linear_i8(x, xs, w, ws, out=out[:4])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(keep, (x, w, out)))
    for call, code in ((lambda: mate.quantize_rows(x[:0].to(torch.bfloat16)), "INVALID_ARG"),
                       (lambda: mate.quantize_rows(x[:, :60].to(torch.bfloat16).contiguous()), "UNSUPPORTED")):
        with pytest.raises(mate.MateError) as e:
            call()
        assert e.value.code == getattr(mate._lib, "MATE_ERR_" + code)


@pytest.mark.parametrize("M", [300, 9001])
def test_products_behind_copies_fills_and_other_streams(M):
    """Products are launched so that they set themselves up under the call ahead of them. Here that call is
    a copy, a fill, a torch kernel, or ends on another stream (a fork and a join), eager and captured."""
    g = _gen(M)
    codes = lambda *s: torch.randint(-127, 128, s, generator=g, dtype=torch.int8, device="cuda")  # noqa: E731
    x0, x1, w = codes(M, 256), codes(M, 256), codes(520, 256)
    xs, ws = torch.rand(M, generator=g, device="cuda"), torch.rand(520, generator=g, device="cuda")
    x = torch.empty_like(x0)
    s2 = torch.empty_like(xs)
    outs = [torch.empty(M, 520, dtype=torch.float32, device="cuda") for _ in range(5)]
    side = torch.cuda.Stream()
    lin = lambda out, scale=xs, **kw: mate.linear_i8(x, scale, w, ws, out_dtype=torch.float32, out=out, **kw)  # noqa: E731

    def run():
        x.copy_(x0)                       # a copy
        lin(outs[0])
        x.zero_()                         # a fill
        lin(outs[1])
        torch.add(x0, 0, out=x)           # a torch kernel
        torch.mul(xs, 2, out=s2)
        lin(outs[2], s2)
        torch.mul(xs, 3, out=s2)          # two kernels on two streams, joined
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            x.copy_(x1)
            lin(outs[3])                  # and a product on the side stream ahead of the join
        main.wait_stream(side)
        lin(outs[4], s2, addend=outs[3])

    def check():
        torch.cuda.synchronize()
        dot = lambda a, s: mate.linear_i8(a, s, w, ws, out_dtype=torch.float32)  # noqa: E731
        assert torch.equal(outs[0], dot(x0, xs)) and (outs[1] == 0).all()
        assert torch.equal(outs[2], dot(x0, 2 * xs)) and torch.equal(outs[3], dot(x1, xs))
        assert torch.equal(outs[4], mate.linear_i8(x1, 3 * xs, w, ws, out_dtype=torch.float32, addend=outs[3]))
        assert mate.mate_last_error() == 0

    for _ in range(3):
        run()
        check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(5):
        for o in (x, s2, *outs):
            o.zero_()
        graph.replay()
        check()


@pytest.mark.slow
def test_offsets_past_32_bits():
    """More than 2^32 elements in a call: sampled rows, the last ones among them, against the same rows alone."""
    M, C = 2 ** 20 + 3, 4104
    rows = torch.tensor([0, 1, 2 ** 19 - 1, 2 ** 19 + 5, M - 2, M - 1], device="cuda")
    g = _gen(1)
    x = torch.empty(M, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    z = torch.empty_like(x).normal_(generator=g)
    w = torch.rand(C, generator=g, device="cuda") + 0.5
    a, b = mate.quantize_rows(x), mate.quantize_rows(x[rows])
    assert torch.equal(a.q[rows], b.q) and torch.equal(a.scale[rows], b.scale)
    a, b = mate.gate_norm_i8(x, z, w, 1368), mate.gate_norm_i8(x[rows], z[rows], w, 1368)
    assert torch.equal(a.q[rows], b.q) and torch.equal(a.scale[rows], b.scale)
    (r, h), (rr, hh) = (mate.block_norm(u[None], v[None], w_post=w, h_dtype=torch.int8) for u, v in ((x, z), (x[rows], z[rows])))
    assert torch.equal(r[0, rows], rr[0]) and torch.equal(h.q[0, rows], hh.q[0]) and torch.equal(h.scale[0, rows], hh.scale[0])
    del x, z, a, r, h
    K = 64
    q = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8, device="cuda")
    wq = torch.randint(-127, 128, (C, K), generator=g, dtype=torch.int8, device="cuda")
    s = torch.rand(M, generator=g, device="cuda")
    out = mate.linear_i8(q, s, wq, w)
    assert torch.equal(out[rows], mate.linear_i8(q[rows], s[rows], wq, w))
    assert torch.equal(mate.linear_i8(q, s, wq, w, addend=out, out=out)[rows], mate.linear_i8(q[rows], s[rows], wq, w, addend=mate.linear_i8(q[rows], s[rows], wq, w)))
    del out
    torch.cuda.empty_cache()
    assert mate.mate_last_error() == 0
