"""Tensors that do not hold what a call would read or write are refused before anything is launched:
block() and stack() hand the entries below a user's weights."""
import pytest
import torch

import workloads
from gpu_util import to_dev

pytestmark = pytest.mark.gpu

mate = pytest.importorskip("linear_complexity_video_b200")

D = 256


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mate.load()


def _layer():
    cfg = workloads.CONFIGS["512p-17s"].with_(T=8, H=16, W=16, nheads=8, attn_heads=2, review=None)
    spec = dict(scan_mode=cfg.modes[0], review_pool=cfg.review, chunk=cfg.chunk, nheads=cfg.nheads, headdim=cfg.headdim,
                ngroups=cfg.ngroups, dstate=cfg.dstate, attn_heads=cfg.attn_heads, attn_dim=cfg.attn_dim, Tw=cfg.Tw,
                Sw=cfg.Sw, shift=cfg.shift)
    return to_dev(workloads.generate_block(cfg, seed=1, d_model=D)), spec


@pytest.mark.parametrize("eight", [False, True], ids=["bf16", "i8"])
def test_block_refuses_weights_that_are_too_short(eight):
    w, spec = _layer()
    u = w["u"]
    make = mate.quantize_block if eight else dict
    keep = mate.block(u, make(w), **spec)
    for name in ("w_in", "conv_w", "conv_b", "dt_bias", "A", "D", "norm_w", "w_q", "w_k", "w_v", "w_ma", "w_te"):
        t = w[name]
        cuts = [t[:-8].contiguous() if t.shape[0] > 8 else t[:-1].contiguous()]
        if name.startswith("w_"):
            cuts.append(t[:, :-64].contiguous())
        for cut in cuts:
            # a shorter w_q leaves another head width, and w_ma's rows are the model width: shapes of another block
            with pytest.raises((ValueError, RuntimeError)):
                mate.block(u, make({**w, name: cut}), **spec)
    assert torch.equal(mate.block(u, make(w), **spec), keep)
    assert mate.mate_last_error() == 0


def test_entries_refuse_tensors_that_are_too_short():
    w, spec = _layer()
    z, x, dt, B, C = mate.frontend(w["u"], w["w_in"], w["conv_w"], w["conv_b"], w["dt_bias"], spec["scan_mode"], 8,
                                   spec["headdim"], spec["ngroups"], spec["dstate"])
    scan = dict(x=x, dt=dt, A=w["A"], B=B, C=C, D=w["D"])
    for kw in (dict(dt=dt[:, 1:].contiguous()), dict(A=w["A"][1:]), dict(D=w["D"][:7]), dict(C=C[:, :7].contiguous()),
               dict(out=x[:, 1:].contiguous()), dict(out=torch.empty_like(x, dtype=torch.float32))):
        with pytest.raises(ValueError):
            mate.bissd(**{**scan, **kw}, scan_mode=0, chunk=spec["chunk"])
    q = torch.zeros(1, 8, 16, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    for args, kw in (((q, q[:, 1:].contiguous(), q), {}), ((q, q, q[..., :1, :].contiguous()), {}),
                     ((q, q, q), dict(out=q[:, 1:].contiguous()))):
        with pytest.raises(ValueError):
            mate.tesa(*args, 2, 8, **kw)
    a, w = (torch.zeros(n, 256, dtype=torch.bfloat16, device="cuda") for n in (40, 64))
    short, ones = torch.zeros(39, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(256, device="cuda")
    for call in (lambda: mate.linear(a, w[:, :192].contiguous()), lambda: mate.linear(a, w, out=short),
                 lambda: mate.compose(a, a, w, w[:, :64].contiguous()), lambda: mate.compose(a, a, w, w[:32]),
                 lambda: mate.compose(a, a, w, w, out=short),
                 lambda: mate.gate_norm(a, a, ones, 256, out=a[:39].clone())):
        with pytest.raises(ValueError):
            call()
    assert mate.linear(a, w).shape == (40, 64)
