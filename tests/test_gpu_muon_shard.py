"""GPU tests of MuonShardStep's refusals and of what it leaves alone."""
import numpy as np
import pytest
import torch

import muon_ref as R
from gpu_util import dev, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def new(Z, S=64, grad=None, matrices=((0, 8, 8),), **kw):
    g = torch.Generator(device=dev()).manual_seed(S)
    p0 = torch.randn(S, generator=g, device=dev())
    return Z.MuonShardStep(S, 1, Z.ZERO_F32 if grad is None else grad, p0, list(matrices), **{"lr": 0.1, **kw})


def test_replicas_of_another_type_are_refused(Z):
    """Of the same size too: their bits would be read as what they are not."""
    t = torch.ones(64, device=dev())
    for grad, bad in ((Z.ZERO_BF16, t.half()), (Z.ZERO_BF16, t), (Z.ZERO_BF16_WIRE, t.half()), (Z.ZERO_F32, t.int()),
                      (Z.ZERO_F32, t.bfloat16()), (Z.ZERO_BF16, t.to(torch.uint8))):
        step = new(Z, grad=grad)
        with pytest.raises(Z.ZeroError, match="a replica of"):
            step.step([bad])
        assert step.t == 0 and bool((step.m == 0).all())
    # bf16 and its bit patterns are the same
    bits = [new(Z, grad=Z.ZERO_BF16) for _ in range(2)]
    bits[0].step([t.bfloat16()])
    bits[1].step([t.bfloat16().view(torch.int16)])
    assert torch.equal(bits[0].master, bits[1].master) and bits[0].t == 1
