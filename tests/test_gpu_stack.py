"""The token mixer in 8 bits (block() with quantize_block's weights) and residual layers of it
(stack()), as programs run the 8-bit operators and the norms together.

The block is checked stage by stage, each against float64 fed the GPU's own inputs to it: the
8-bit stages within the bounds of plain64.py, the bf16 ones (the front-end after its products,
the scan, the attention) within the bf16 bound of the other parity tests."""
import numpy as np
import pytest
import torch

import oracle
import plain64
import workloads
from gpu_util import TOL, host64, rel_err, to_dev

pytestmark = pytest.mark.gpu

mate = pytest.importorskip("linear_complexity_video_b200")

D = 256


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mate.load()


def _cfg(name, **kw):
    return workloads.CONFIGS[name].with_(**{**dict(T=8, H=16, W=16, nheads=8, attn_heads=2), **kw})


def _spec(cfg):
    return dict(scan_mode=cfg.modes[0], review_pool=cfg.review, chunk=cfg.chunk, nheads=cfg.nheads,
                headdim=cfg.headdim, ngroups=cfg.ngroups, dstate=cfg.dstate, attn_heads=cfg.attn_heads,
                attn_dim=cfg.attn_dim, Tw=cfg.Tw, Sw=cfg.Sw, shift=cfg.shift)


def _value(c):
    return host64(c.q) * host64(c.scale)[..., None]


def _check_linear(got, x, w, addend=None):
    x2 = x.q.reshape(-1, x.q.shape[-1])
    ref, tol = plain64.linear(host64(x2), host64(x.scale).reshape(-1), host64(w.q), host64(w.scale), None, addend)
    limit = tol + plain64.HALF_STEP["bf16"] * (np.abs(ref) + tol)
    off = np.abs(host64(got).reshape(ref.shape) - ref)
    assert (off <= limit).all(), float((off / limit).max())


@pytest.mark.parametrize("codes_in", [False, True], ids=["bf16-in", "codes-in"])
@pytest.mark.parametrize("name,kw", [("512p-17s", {}), ("512p-68s", {}), ("768p-17s", dict(T=5, H=8, W=24))])
def test_block_i8_stages(name, kw, codes_in):
    cfg = _cfg(name, **kw)
    p = workloads.generate_block(cfg, seed=3, d_model=D)
    dev = to_dev(p)
    w8 = mate.quantize_block(dev)
    u = mate.quantize_rows(dev["u"]) if codes_in else dev["u"]
    out, mid = mate.block(u, w8, keep=True, **_spec(cfg))
    assert torch.equal(out, mate.block(u, w8, **_spec(cfg))) or cfg.review  # (review sums by atomics)
    assert mate.mate_last_error() == 0
    o = oracle.get()
    q, s = plain64.codes(p["u"].double().numpy())
    assert np.array_equal(host64(mid["u"].q), q)
    for n in ("w_in", "w_q", "w_k", "w_v", "w_ma", "w_te"):
        assert np.array_equal(host64(w8[n].q), plain64.codes(p[n].double().numpy())[0])
    ref = o.frontend(_value(mid["u"]), _value(w8["w_in"]), p["conv_w"], p["conv_b"], p["dt_bias"], cfg.modes[0],
                     cfg.nheads, cfg.headdim, cfg.ngroups, cfg.dstate)
    for n, r in zip("z x dt B C".split(), ref):
        assert rel_err(host64(mid[n]), r) <= TOL["bf16"], n
    y = o.bissd(host64(mid["x"]), host64(mid["dt"]), p["A"], host64(mid["B"]), host64(mid["C"]), p["D"], cfg.modes[0],
                cfg.review)
    assert rel_err(host64(mid["y"]), y) <= TOL["bf16"], "bi-SSD"
    d_inner, te = cfg.nheads * cfg.headdim, cfg.attn_heads * cfg.attn_dim
    plain64.check_codes(host64(mid["y_ma"].q).reshape(-1, d_inner), host64(mid["y_ma"].scale).reshape(-1),
                        *plain64.gate_norm(host64(mid["y"]).reshape(-1, d_inner), host64(mid["z"]).reshape(-1, d_inner),
                                           p["norm_w"].double(), d_inner // cfg.ngroups, 1e-5))
    for n, wn in (("q", "w_q"), ("k", "w_k"), ("v", "w_v")):
        _check_linear(mid[n], mid["u"], w8[wn])
    t = o.tesa(host64(mid["q"]), host64(mid["k"]), host64(mid["v"]), cfg.Tw, cfg.Sw, cfg.shift)
    assert rel_err(host64(mid["y_te"]), t) <= TOL["bf16"], "TESA"
    assert np.array_equal(host64(mid["c_te"].q).reshape(-1, te), plain64.codes(host64(mid["y_te"]).reshape(-1, te))[0])
    _check_linear(mid["te"], mid["c_te"], w8["w_te"])
    _check_linear(out, mid["y_ma"], w8["w_ma"], addend=host64(mid["te"]).reshape(-1, D))


def test_block_i8_near_the_exact_chain():
    """The 8-bit block against the whole chain in float64 from u. A row of a few hundred normal
    values has its largest near 3.3 sigma, so a code's error, uniform over max / 127, has an rms of
    0.0075 sigma: 0.011 per product for its two factors, about 0.02 through the scan (x, B and C
    enter as a product), 0.03 with the composition's own. The bound is three times that."""
    cfg = _cfg("512p-17s")
    p = workloads.generate_block(cfg, seed=3, d_model=D)
    dev = to_dev(p)
    got = host64(mate.block(dev["u"], mate.quantize_block(dev), **_spec(cfg))).reshape(-1, D)
    o = oracle.get()
    z, x, dt, B, C = o.frontend(p["u"], p["w_in"], p["conv_w"], p["conv_b"], p["dt_bias"], cfg.modes[0], cfg.nheads,
                                cfg.headdim, cfg.ngroups, cfg.dstate)
    y = o.bissd(x, dt, p["A"], B, C, p["D"], cfg.modes[0], cfg.review)
    d_inner, te = cfg.nheads * cfg.headdim, cfg.attn_heads * cfg.attn_dim
    y_ma = o.gate_norm(y.reshape(-1, d_inner), z.reshape(-1, d_inner), p["norm_w"], d_inner, 1e-5)
    u64 = p["u"].double().numpy().reshape(-1, D)
    qkv = [(u64 @ p[n].double().numpy().T).reshape(cfg.batch, cfg.T, cfg.H, cfg.W, cfg.attn_heads, cfg.attn_dim)
           for n in ("w_q", "w_k", "w_v")]
    y_te = o.tesa(*qkv, cfg.Tw, cfg.Sw, cfg.shift)
    ref = o.compose(y_ma, y_te.reshape(-1, te), p["w_ma"], p["w_te"])
    assert np.linalg.norm(got - ref) <= 0.1 * np.linalg.norm(ref)


def _layers(cfg, eight, n=3):
    layers = []
    for i in range(n):
        p = workloads.generate_layer(cfg, seed=10 * i, d_model=D)
        d = to_dev({k: v for k, v in p.items() if k != "u"})
        mod = mate.modulation(d["c"], mate.quantize_rows(d["w_mod"]), d["b_mod"])
        ref, tol = plain64.linear(*plain64.codes(p["c"].double().numpy()), *plain64.codes(p["w_mod"].double().numpy()),
                                  p["b_mod"].double())
        # the scales' own roundings: 2 u of the product more
        assert (np.abs(host64(mod) - ref) <= tol * 2 + plain64.U * np.abs(ref)).all()
        layers.append((mate.quantize_block(d) if eight else d, mod,
                       dict(scan_mode=i % 4, shift=(0, 0, 0) if i % 2 else cfg.shift)))
    return layers


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("eight", [False, True], ids=["bf16", "i8"])
def test_stack_equals_its_parts(eight, norm):
    """With an fp32 residual stream nothing is rounded between the norm after a layer and the one
    before the next, so the stack is its parts called one by one, bit for bit."""
    cfg = _cfg("512p-17s", batch=2, T=4, review=None)
    layers = _layers(cfg, eight)
    x0 = torch.randn(2, 4, 16, 16, D, generator=torch.Generator().manual_seed(1)).cuda()
    keep = x0.clone()
    got = mate.stack(x0, layers, norm=norm, residual_scale=0.875, **_spec(cfg))
    assert torch.equal(x0, keep)
    x = x0
    for w, mod, over in layers:
        shift, scale, gate = (m.contiguous() for m in mod.split(D, 1))
        _, h = mate.block_norm(x, w_pre=w["w_pre"], scale=scale, shift=shift, norm=norm,
                               h_dtype=torch.int8 if eight else torch.bfloat16)
        y = mate.block(h, w, **{**_spec(cfg), **over})
        first, _ = plain64.block_norm(host64(x).reshape(2, -1, D), host64(y).reshape(2, -1, D), host64(w["w_post"]),
                                      host64(gate), 0.875, norm)
        x, _ = mate.block_norm(x, y, w_post=w["w_post"], gate=gate, residual_scale=0.875, norm=norm, h_dtype=None)
        off = np.abs(host64(x).reshape(2, -1, D) - first[0])
        assert (off <= first[1] + plain64.U * np.abs(first[0])).all()
    assert torch.equal(got, x)
    assert mate.mate_last_error() == 0


@pytest.mark.parametrize("eight", [False, True], ids=["bf16", "i8"])
def test_stack_captured(eight):
    cfg = _cfg("512p-17s", T=4, review=None)
    layers = _layers(cfg, eight, n=2)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(1, 4, 16, 16, D, generator=g).to(torch.bfloat16).cuda()
    mate.stack(x, layers, **_spec(cfg))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mate.stack(x, layers, **_spec(cfg))
    for _ in range(2):
        new = torch.randn(1, 4, 16, 16, D, generator=g).to(torch.bfloat16).cuda()
        x.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mate.stack(new, layers, **_spec(cfg)))


def test_stack_on_a_stream_and_empty():
    cfg = _cfg("512p-17s", T=4, review=None)
    layers = _layers(cfg, True, n=1)
    x = torch.randn(1, 4, 16, 16, D, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    want = mate.stack(x, layers, **_spec(cfg))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = mate.stack(x, layers, stream=st, **_spec(cfg))
    st.synchronize()
    assert torch.equal(got, want)
    assert mate.stack(x, []) is x


def test_block_refuses_mixed_weights():
    cfg = _cfg("512p-17s", T=4)
    dev = to_dev(workloads.generate_block(cfg, d_model=D))
    w8 = mate.quantize_block(dev)
    with pytest.raises(ValueError, match="none"):
        mate.block(dev["u"], {**w8, "w_q": dev["w_q"]}, **_spec(cfg))
    with pytest.raises(ValueError, match="8-bit too"):
        mate.block(mate.quantize_rows(dev["u"]), dev, **_spec(cfg))
