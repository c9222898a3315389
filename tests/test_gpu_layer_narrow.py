"""Few rows through few outputs with a long reduction, on both sides of the border between
the kernel that streams the weights and split tiles."""
import numpy as np
import pytest
import torch

import layer_ref as R
from gpu_util import dev, say
from test_gpu_layer import BF, F32, LAYOUTS, Mat, close, inp, rand, rng_of, w64, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("rows,long,narrow", [(1, 50257, 64), (1, 9600, 16), (1, 10400, 16), (4, 16384, 40), (8, 9000, 200),
                                              (16, 7000, 65), (16, 8192, 130), (2, 30000, 1), (3, 12345, 1000)])
def test_long_reductions_of_few_rows(Z, rows, long, narrow, layout):
    rng = rng_of((91, rows, long, narrow, layout))
    for place in ((0, 0), (3, 1)):
        x, w = inp(rng, rows, long, pad_ld=place[0], shift=place[1]), weight(rng, long, narrow, layout, place)
        b = torch.from_numpy(rand(rng, narrow)).to(dev()).to(BF)
        y, z = Mat(rows, narrow, BF, ld=narrow + 5), Mat(rows, narrow, BF, ld=narrow + 8)
        say("long reduction of few rows", rows, long, narrow, layout, place)
        Z.zero_linear_forward(x.t, w.t, b, w_layout=layout, act=2, y=y.t, preact=z.t)
        want, err, wz, ez = R.linear_forward(x.f64(), w64(w, layout), b.cpu().double().numpy(), act_name="gelu")
        close("y", y.t, want, err)
        close("z", z.t, wz, ez)
        assert y.intact_outside() and z.intact_outside()
        # the weights' other way round: a layer of `narrow` inputs and `long` outputs
        w = weight(rng, narrow, long, layout, place)
        dz, zz = inp(rng, rows, long, pad_ld=place[0], shift=place[1]), inp(rng, rows, narrow)
        dx = Mat(rows, narrow, F32, ld=narrow + 3)
        Z.zero_linear_grad_input(dz.t, w.t, w_layout=layout, act=3, preact=zz.t, dx=dx.t)
        want, err = R.linear_grad_input(dz.f64(), w64(w, layout), act_name="silu", z=zz.f64(), out="f32")
        close("dx", dx.t, want, err)
        assert dx.intact_outside()
