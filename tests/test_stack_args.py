"""Arguments that stack() refuses before it computes anything (CPU only)."""
import pytest
import torch

import linear_complexity_video_b200 as mate

SPEC = dict(scan_mode=0, review_pool=None, chunk=256, nheads=8, headdim=64, ngroups=1, dstate=64, attn_heads=2,
            attn_dim=64, Tw=2, Sw=4, shift=(0, 0, 0))


@pytest.mark.parametrize("over,more", [({}, dict(keep=True)), (dict(keep=True), {}), (dict(keep=False), {}),
                                       (dict(stream=0), {})])
def test_stack_refuses_keep_and_streams_of_layers(over, more):
    """A layer with its intermediate tensors is no layer's input, and a layer on a stream of its own would
    run beside the norms it hands over to."""
    x, mod = torch.zeros(1, 2, 4, 4, 64), torch.zeros(1, 192)
    for layers in ([({}, mod, over)], [({}, mod), ({}, mod, over)]):
        with pytest.raises(ValueError, match="keep"):
            mate.stack(x, layers, **SPEC, **more)


def test_stack_refuses_another_modulation():
    x = torch.zeros(2, 2, 4, 4, 64)
    for shape in ((1, 192), (2, 128), (192,)):
        with pytest.raises(ValueError, match="mod must be"):
            mate.stack(x, [({}, torch.zeros(shape))], **SPEC)
