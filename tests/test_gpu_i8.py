"""The 8-bit operators (mate_quant_rows_fwd, mate_linear_i8_fwd, mate_gate_norm_i8_fwd) against
plain float64 (plain64.py, which derives the bounds). Row codes of bf16 are compared bit for bit:
they are the correctly rounded values."""
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
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------- row quantisation
@pytest.mark.parametrize("M,K", [(1, 8), (1, 2560), (2, 1280), (3, 1288), (5, 2568), (301, 64), (37, 5120), (9, 5128),
                                 (4, 10240), (3, 20480), (1155, 2560), (33, 20472)])
def test_quantize_rows_bit_exact(M, K):
    g = _gen(M * 7 + K)
    x = (torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g) * 4)).to(torch.bfloat16)
    got = mate.quantize_rows(x.cuda())
    q, s = plain64.codes(x.double().numpy())
    assert np.array_equal(host64(got.q), q)
    assert (np.abs(host64(got.scale) - s) <= plain64.U * s).all()


def test_quantize_rows_ties_and_borders():
    """Every bf16 magnitude of two binades against every significand of the largest one: each tie
    (127 / 2 at half the largest, and all of them where it is 254 x 2^k) goes to the even code."""
    sig = torch.arange(128, 256, dtype=torch.float32)
    small = torch.cat([sig / 2 ** k for k in range(1, 10)])
    rows = []
    for a in sig:
        r = torch.cat([small, -small, torch.zeros(2)])
        r = r[: r.numel() // 8 * 8]
        r[r.abs() > a] = 0
        r[0] = a
        rows.append(r)
    x = torch.stack(rows).to(torch.bfloat16)
    got = mate.quantize_rows(x.cuda())
    q, _ = plain64.codes(x.double().numpy())
    assert np.array_equal(host64(got.q), q)


def test_quantize_rows_extreme_rows():
    big, tiny = torch.finfo(torch.bfloat16).max, 2.0 ** -133  # the smallest bf16 subnormal
    x = torch.zeros(10, 264, dtype=torch.float32)
    x[1, 3] = tiny
    x[2] = torch.linspace(-1, 1, 264) * 2.0 ** -126
    x[3] = torch.linspace(-1, 1, 264) * 2.0 ** -101
    x[4] = torch.linspace(-1, 1, 264) * big
    x[5, 7], x[5, 0] = float("inf"), 1.0
    x[6, 263], x[6, 0] = float("-inf"), 1.0
    x[7, 100], x[7, 0] = float("nan"), 1.0
    x[8, 5], x[8, 6] = float("nan"), float("inf")
    x[9] = -big
    x = x.to(torch.bfloat16)
    got = mate.quantize_rows(x.cuda())
    q, s = plain64.codes(x.double().numpy())
    assert np.array_equal(host64(got.q), q)
    gs = host64(got.scale)
    assert np.isnan(gs[5:9]).all() and np.isfinite(gs[:5]).all()
    fin = ~np.isnan(s)
    assert (np.abs(gs - s)[fin] <= plain64.U * s[fin] + 2.0 ** -150).all()  # a subnormal scale: half its step


def test_quantize_rows_writes_its_rows_only():
    x = torch.randn(7, 72, generator=_gen(0)).to(torch.bfloat16).cuda()
    q = torch.full((9, 72), 99, dtype=torch.int8, device="cuda")
    s = torch.full((9,), 7.0, device="cuda")
    mate.mate_quant_rows_fwd(x, q, s, mate.api.mate_quant_dims(7, 72, 1))
    assert (q[7:] == 99).all() and (s[7:] == 7).all() and (q[:7] != 99).any()


# ---------------------------------------------------------------- linear layer
def _linear_inputs(M, K, N, seed, dtype=torch.bfloat16, extreme=False):
    g = _gen(seed)
    xq = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8)
    if extreme:  # the largest sums there are, of either sign
        xq = torch.full((M, K), 127, dtype=torch.int8)
        xq[::2] = -127
        wq = torch.full((N, K), 127, dtype=torch.int8)
    xs = torch.rand(M, generator=g) + 0.01
    ws = (torch.rand(N, generator=g) + 0.01) / K
    bias = torch.randn(N, generator=g)
    addend = torch.randn(M, N, generator=g).to(dtype)
    return xq, xs, wq, ws, bias, addend


def _check_linear(got, xq, xs, wq, ws, bias, addend, dtype):
    ref, tol = plain64.linear(xq, xs, wq, ws, bias, None if addend is None else addend.double())
    half = plain64.HALF_STEP["bf16" if dtype == torch.bfloat16 else "f32"]
    off = np.abs(host64(got) - ref)
    limit = tol + half * (np.abs(ref) + tol)
    assert (off <= limit).all(), float((off / limit).max())


SHAPES = [(1, 16, 8), (1, 2560, 7680), (2, 2560, 264), (7, 80, 40), (16, 2560, 2560), (17, 1296, 1000), (31, 144, 5248),
          (33, 5120, 520), (64, 2560, 80), (65, 2560, 2560), (127, 272, 72), (128, 128, 256), (129, 2576, 264),
          (200, 7680, 136), (255, 400, 2560), (257, 128, 512), (300, 2560, 2560), (513, 1040, 776), (1155, 2560, 2560),
          (1155, 48, 10448), (2500, 5120, 264), (4097, 64, 64),
          # the pairs' kernel, ragged in every direction, with one to eleven tile columns
          (1921, 144, 2312), (4225, 272, 2568), (9000, 400, 2504), (12800, 128, 1048), (513, 2576, 10440)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear_i8(M, K, N, dtype):
    xq, xs, wq, ws, bias, addend = _linear_inputs(M, K, N, seed=M + K + N, dtype=dtype)
    use_bias, use_add = (M + N // 8) % 2 == 0, (M + K // 16) % 3 == 0
    bias, addend = bias if use_bias else None, addend if use_add else None
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = mate.linear_i8(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), bias=d(bias), addend=d(addend), out_dtype=dtype)
    assert mate.mate_last_error() == 0
    _check_linear(got, xq, xs, wq, ws, bias, addend, dtype)


@pytest.mark.parametrize("M,K,N", [(3, 131072, 16), (130, 66048, 264)])
def test_linear_i8_largest_sums_are_exact(M, K, N):
    """127 * 127 * 131,072 = 2,114,060,288 is the largest sum: it must not wrap."""
    xq, _, wq, _, _, _ = _linear_inputs(M, K, N, 0, extreme=True)
    one = lambda n: torch.ones(n)  # noqa: E731
    got = mate.linear_i8(xq.cuda(), one(M).cuda(), wq.cuda(), one(N).cuda(), out_dtype=torch.float32)
    ref = torch.full((M, N), 127.0 * 127.0 * K, dtype=torch.float64)
    ref[::2] *= -1
    assert torch.equal(got.cpu(), ref.float())


@pytest.mark.parametrize("M,K,N", [(5, 320, 264), (300, 320, 264), (20000, 128, 136)])
def test_linear_i8_addend_in_place_and_rows_behind(M, K, N):
    xq, xs, wq, ws, bias, addend = _linear_inputs(M, K, N, seed=3)
    buf = torch.full((M + 3, N), 5.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:M]
    out.copy_(addend)
    mate.linear_i8(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), addend=out, out=out)
    _check_linear(out, xq, xs, wq, ws, None, addend, torch.bfloat16)
    assert (buf[M:] == 5).all()


def test_linear_i8_is_reproducible_and_keeps_nan_rows():
    xq, xs, wq, ws, _, _ = _linear_inputs(70, 4096, 2560, seed=5)
    xs[3] = float("nan")
    xq[3] = 0
    xs[4] = 0.0
    d = [t.cuda() for t in (xq, xs, wq, ws)]
    a, b = mate.linear_i8(*d), mate.linear_i8(*d)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert torch.isnan(a[3]).all() and (a[4] == 0).all() and torch.isfinite(a[5:]).all()


def test_leading_shapes():
    xq, xs, wq, ws, _, _ = _linear_inputs(24, 64, 40, seed=6)
    d = [t.cuda() for t in (xq, xs, wq, ws)]
    a = mate.linear_i8(*d)
    b = mate.linear_i8(d[0].view(2, 3, 4, 64), d[1].view(2, 3, 4), d[2], d[3])
    assert b.shape == (2, 3, 4, 40) and torch.equal(a, b.view(24, 40))
    # a single row without a leading dimension
    one = mate.linear_i8(d[0][5], d[1][5], d[2], d[3])
    assert one.shape == (40,) and torch.equal(one, a[5])
    x = torch.randn(3, 5, 64, generator=_gen(1)).to(torch.bfloat16).cuda()
    c, r = mate.quantize_rows(x), mate.quantize_rows(x[1, 2])
    assert c.scale.shape == (3, 5) and r.scale.shape == ()
    assert torch.equal(c.q[1, 2], r.q) and torch.equal(c.scale[1, 2], r.scale)


def test_refusals_on_the_device():
    xq, xs, wq, ws, bias, addend = [t.cuda() for t in _linear_inputs(8, 64, 40, seed=7)]
    ok = dict(x_q=xq, x_scale=xs, w_q=wq, w_scale=ws)
    for kw in (dict(x_q=xq.float()), dict(x_q=xq[:, :32]), dict(x_q=xq.t()), dict(x_scale=xs[:4]), dict(x_scale=xs.double()),
               dict(x_scale=xs[:, None]), dict(w_q=wq[0]), dict(w_scale=ws[:8]), dict(bias=bias[:8]), dict(bias=bias.half()),
               dict(addend=addend[:4]), dict(addend=addend.float()), dict(out_dtype=torch.float16), dict(x_q=None),
               dict(out=torch.empty(8, 48, dtype=torch.bfloat16, device="cuda")), dict(x_scale=xs.cpu())):
        with pytest.raises(ValueError):
            mate.linear_i8(**{**ok, **kw})
    # no rows; rows of codes off the 16-byte boundary; an output over an input
    for kw in (dict(x_q=xq[:0], x_scale=xs[:0]), dict(x_q=torch.empty(8 * 64 + 8, dtype=torch.int8, device="cuda")[8:].view(8, 64)),
               dict(out=xq.view(torch.bfloat16).flatten()[:1].expand(1), x_q=xq[:1], x_scale=xs[:1], w_q=wq[:1], w_scale=ws[:1])):
        with pytest.raises((mate.MateError, ValueError)):
            mate.linear_i8(**{**ok, **kw})
    with pytest.raises(mate.MateError):
        mate.quantize_rows(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(mate.MateError):
        mate.quantize_rows(torch.zeros(4, 60, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.slow
def test_linear_i8_in_proj_131k():
    """The block's largest product: 64 sampled rows, and outputs past 2^31 bytes."""
    M, K, N = 131072, 2560, 10448
    g = torch.Generator(device="cuda").manual_seed(1)
    xq = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8, device="cuda")
    wq = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8, device="cuda")
    xs = torch.rand(M, generator=g, device="cuda") + 0.01
    ws = (torch.rand(N, generator=g, device="cuda") + 0.01) / K
    got = mate.linear_i8(xq, xs, wq, ws)
    assert mate.mate_last_error() == 0
    rows = torch.randperm(M, generator=_gen(2))[:62].tolist() + [0, M - 1]
    _check_linear(got[rows], xq[rows].cpu(), xs[rows].cpu(), wq.cpu(), ws.cpu(), None, None, torch.bfloat16)


# ---------------------------------------------------------------- gated norm, 8-bit output
@pytest.mark.parametrize("M,C,group", [(1, 8, 8), (3, 64, 16), (37, 5120, 5120), (5, 5120, 2560), (2, 8192, 8192),
                                       (9, 1032, 344), (700, 1024, 1024)])
def test_gate_norm_i8(M, C, group):
    g = _gen(C + M)
    y, z = (torch.randn(M, C, generator=g).to(torch.bfloat16) for _ in range(2))
    w = 1 + torch.randn(C, generator=g) / 10
    got = mate.gate_norm_i8(y.cuda(), z.cuda(), w.cuda(), group, 1e-5)
    ref, tol = plain64.gate_norm(y.double(), z.double(), w.double(), group, 1e-5)
    plain64.check_codes(host64(got.q), host64(got.scale), ref, tol)


def test_gate_norm_i8_zero_and_not_finite_rows():
    y = torch.ones(4, 64, dtype=torch.bfloat16)
    z = torch.ones(4, 64, dtype=torch.bfloat16)
    y[1] = 0
    y[2, 5] = float("nan")
    y[3, 63] = float("inf")
    got = mate.gate_norm_i8(y.cuda(), z.cuda(), torch.ones(64).cuda(), 64)
    q, s = host64(got.q), host64(got.scale)
    assert (q[0] == 127).all() and (q[1:] == 0).all()
    assert s[1] == 0 and np.isnan(s[2:]).all()


# ---------------------------------------------------------------- together, and as programs run them
def test_quantised_linear_near_the_exact_product():
    """quantize_rows of both sides and the product, against x w^T in float64. Each factor is off
    by at most half its row's scale: |dx| <= sx/2, |dw| <= sw/2 (times 1 + 2^-20 for the scales'
    roundings), so |sum| moves by at most (sum|w| sx + sum|x| sw)/2 + K sx sw/4."""
    g = _gen(11)
    x = torch.randn(45, 2560, generator=g).to(torch.bfloat16)
    w = (torch.randn(264, 2560, generator=g) / 50).to(torch.bfloat16)
    cx, cw = mate.quantize_rows(x.cuda()), mate.quantize_rows(w.cuda())
    got = host64(mate.linear_i8(*cx, *cw, out_dtype=torch.float32))
    xd, wd = x.double().numpy(), w.double().numpy()
    sx, sw = np.abs(xd).max(1)[:, None] / 127, np.abs(wd).max(1)[None] / 127
    ref = xd @ wd.T
    limit = (np.abs(wd).sum(1)[None] * sx + np.abs(xd).sum(1)[:, None] * sw) / 2 + 2560 * sx * sw / 4
    assert (np.abs(got - ref) <= limit * (1 + 2.0 ** -18)).all()
    assert np.abs(got - ref).max() <= 0.05 * np.abs(ref).max()  # and in effect far nearer


def _chain(x, w, y, z, wn):
    c = mate.quantize_rows(x)
    a = mate.linear_i8(*c, *w)
    n = mate.gate_norm_i8(y, z, wn, 64)
    _, h = mate.block_norm(a.view(1, *a.shape), h_dtype=torch.int8)
    return a, n.q, n.scale, h.q, h.scale


def _chain_inputs(M, seed):
    g = _gen(seed)
    x = torch.randn(M, 256, generator=g).to(torch.bfloat16).cuda()
    y, z = (torch.randn(M, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    return x, y, z


@pytest.mark.parametrize("M", [3, 400, 20000])
def test_captured_and_replayed(M):
    """One capture, replayed on new inputs: the results of the eager calls, bit for bit; the
    error word still reads clean."""
    w = mate.quantize_rows(torch.randn(136, 256, generator=_gen(1)).to(torch.bfloat16).cuda())
    wn = torch.ones(128, device="cuda")
    x, y, z = _chain_inputs(M, 2)
    _chain(x, w, y, z, wn)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _chain(x, w, y, z, wn)
    for seed in (3, 4):
        new = _chain_inputs(M, seed)
        for dst, src in zip((x, y, z), new):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, _chain(*new[:1], w, *new[1:], wn)):
            assert torch.equal(a, b)
    assert mate.mate_last_error() == 0


@pytest.mark.parametrize("M", [700, 9001])
def test_two_streams_at_once(M):
    w = mate.quantize_rows(torch.randn(520, 256, generator=_gen(1)).to(torch.bfloat16).cuda())
    wn = torch.ones(128, device="cuda")
    ins = [_chain_inputs(M, s) for s in (5, 6)]
    want = [_chain(i[0], w, i[1], i[2], wn) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [[], []]
    for _ in range(5):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(_chain(ins[k][0], w, ins[k][1], ins[k][2], wn))
    torch.cuda.synchronize()
    for k in range(2):
        for outs in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[k]))


@pytest.mark.parametrize("M", [5, 300, 6000])
def test_reused_buffers_keep_stream_order(M):
    """Products and quantisations that read and overwrite the same few buffers, forty calls without a
    wait between them: what waiting after every call gives, bit for bit (the products are launched
    so that they may set themselves up before the call ahead of them has ended)."""
    g = _gen(M)
    w = [mate.quantize_rows((torch.randn(256, 256, generator=g) / 16).to(torch.bfloat16).cuda()) for _ in range(2)]
    x0 = torch.randn(M, 256, generator=g).to(torch.bfloat16).cuda()

    def run(wait):
        a, b = x0.clone(), torch.empty_like(x0)
        q, s = torch.empty(M, 256, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        dims = mate.api.mate_quant_dims(M, 256, 1)
        for i in range(20):
            mate.mate_quant_rows_fwd(a, q, s, dims)
            wait()
            mate.linear_i8(q, s, *w[i % 2], out=b)
            wait()
            mate.linear_i8(q, s, *w[(i + 1) % 2], addend=b, out=b)
            wait()
            a, b = b, a
        return a

    slow = run(torch.cuda.synchronize)
    fast = run(lambda: None)
    assert torch.equal(slow, fast) and torch.isfinite(fast).all()


def test_two_graphs_of_one_workspace_free_chain():
    """Two captured graphs of the same calls, replayed in turn and on two streams: nothing is shared."""
    w = mate.quantize_rows(torch.randn(520, 256, generator=_gen(1)).to(torch.bfloat16).cuda())
    wn = torch.ones(128, device="cuda")
    ins = [_chain_inputs(m, s) for m, s in ((30, 7), (9001, 8))]
    want = [_chain(i[0], w, i[1], i[2], wn) for i in ins]
    torch.cuda.synchronize()
    graphs = []
    for i in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = _chain(i[0], w, i[1], i[2], wn)
        graphs.append((g, outs))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for (g, _o), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_g, outs), ref in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))


@pytest.mark.parametrize("as_handle", [False, True])
def test_stream_argument(as_handle):
    x = torch.randn(50, 256, generator=_gen(1)).to(torch.bfloat16).cuda()
    w = mate.quantize_rows(torch.randn(64, 256, generator=_gen(2)).to(torch.bfloat16).cuda())
    want = mate.linear_i8(*mate.quantize_rows(x), *w)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    arg = st.cuda_stream if as_handle else st
    got = mate.linear_i8(*mate.quantize_rows(x, stream=arg), *w, stream=arg)
    st.synchronize()
    assert torch.equal(got, want)


def test_several_host_threads():
    import threading

    xq, xs, wq, ws, _, _ = [t.cuda() for t in _linear_inputs(9000, 256, 136, seed=8)]
    x = torch.randn(40, 256, generator=_gen(9)).to(torch.bfloat16).cuda()
    want = (mate.linear_i8(xq, xs, wq, ws), mate.linear_i8(xq[:40], xs[:40], wq, ws), *mate.quantize_rows(x))
    torch.cuda.synchronize()
    got = []

    def work():
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(20):
                r = (mate.linear_i8(xq, xs, wq, ws), mate.linear_i8(xq[:40], xs[:40], wq, ws), *mate.quantize_rows(x))
        st.synchronize()
        got.append(r)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 4 and all(torch.equal(a, b) for r in got for a, b in zip(r, want))
