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


@pytest.mark.parametrize("rows,K,N", [(1, 4096, 1104), (4, 4096, 4096)])
def test_few_aligned_rows_need_no_workspace(Z, rows, K, N):
    """A call without one is served where its rows are on 16 bytes, and where they are not it
    is refused if the sizes ask for one: 4096 elements into 1104 columns are split there
    (4096 * 3.28e-3 is above 6.5 + 9.04 / 3.3), four rows into 4096 are not (4096 * 3.82e-3
    is below 6.5 + 33.6 / 3.3)."""
    need = Z.zero_linear_workspace_bytes(Z.ZERO_LINEAR_FORWARD, Z.ZERO_W_OUT_IN, rows, K, N)
    assert (need > 0) == (N == 1104)
    rng = rng_of((92, rows, K, N))
    x, w = inp(rng, rows, K), weight(rng, K, N, 0, (0, 0))
    y = torch.empty((rows, N), dtype=F32, device=dev())
    none = torch.empty(0, dtype=torch.uint8, device=dev())
    say("no workspace", rows, K, N)
    Z.zero_linear_forward(x.t, w.t, y=y, workspace=none)
    want, err, _, _ = R.linear_forward(x.f64(), w64(w, 0), out="f32")
    close("y", y, want, err)
    odd = weight(rng, K, N, 0, (1, 0))
    if need == 0:
        Z.zero_linear_forward(x.t, odd.t, y=y, workspace=none)
        want, err, _, _ = R.linear_forward(x.f64(), w64(odd, 0), out="f32")
        close("y", y, want, err)
        return
    with pytest.raises(Z.ZeroError, match="workspace_dev"):
        Z.zero_linear_forward(x.t, odd.t, y=y, workspace=none)
