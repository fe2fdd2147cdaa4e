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
