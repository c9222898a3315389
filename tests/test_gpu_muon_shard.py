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
    bits = [new(Z, grad=Z.ZERO_BF16) for _ in range(3)]
    for step, as_type in zip(bits, (BF, torch.int16, torch.uint16)):
        step.step([t.bfloat16().view(as_type)])
        assert torch.equal(step.master, bits[0].master) and step.t == 1


BAD = [dict(lr=-0.1), dict(lr=float("nan")), dict(weight_decay=float("inf")), dict(mu=1.0), dict(steps=0), dict(steps=8),
       dict(eps=0.0), dict(coefficients=(1.0, float("nan"), 0.0)), dict(coefficients=[(1.0, 2.0, 3.0)] * 4),
       dict(scale=lambda r, c: 1e9)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_bad_hyperparameters_are_refused_before_anything_is_written(Z, bad):
    """By the constructor; and where they are set later, by a step that leaves its state as it was."""
    with pytest.raises(Z.ZeroError):
        new(Z, **bad)
    if "scale" in bad:
        return
    step = new(Z)
    g = torch.ones(64, device=dev())
    step.step([g])
    was = step.state_dict()
    for group in (step.hyper, step.momentum_hyper, step.orth):
        group.update({k: v for k, v in bad.items() if k in group})
    with pytest.raises(Z.ZeroError):
        step.step([g])
    torch.cuda.synchronize()
    now = step.state_dict()
    assert torch.equal(was["m"], now["m"]) and torch.equal(was["p"], now["p"]) and now["t"] == 1
    assert torch.equal(step.slot.view(BF), step.master.to(BF))


def test_a_slot_that_is_not_the_shards_is_refused(Z):
    for slot in (torch.zeros(64, dtype=torch.int16), torch.zeros(128, dtype=torch.int16, device=dev())[::2],
                 torch.zeros(63, dtype=torch.int16, device=dev()), torch.zeros(64, dtype=torch.float16, device=dev()),
                 torch.zeros(8, 8, dtype=BF, device=dev())):
        with pytest.raises(Z.ZeroError, match="slot is"):
            new(Z, slot=slot)
    mine = torch.zeros(64, dtype=BF, device=dev())
    step = new(Z, slot=mine)
    step.step([torch.ones(64, device=dev())])
    assert step.slot is mine and torch.equal(mine, step.master.to(BF))


@pytest.mark.parametrize("given", [True, False])
def test_what_no_matrix_holds_is_left_alone(Z, given):
    """A norm and a bias between the matrices and an embedding behind them, with weight decay:
    master copy and slot keep their bits, also where another optimizer has changed them in
    between; the matrices are updated as in a shard of their own."""
    S = 2000
    mats = [(0, 10, 40), (400, 10, 40), (900, 20, 25), (1408, 12, 16)]
    slot = torch.zeros(S, dtype=torch.int16, device=dev()) if given else None
    step = new(Z, S, matrices=mats, weight_decay=0.1, slot=slot)
    inside = torch.zeros(S, dtype=torch.bool, device=dev())
    for o, r, c in mats:
        inside[o:o + r * c] = True
    inside[1400:1408] = True                    # padding between the last two
    assert step.runs == [(0, 800), (900, 1600)]
    rest = ~inside
    p0 = step.master.clone()
    say("a shard of matrices and others")
    g = torch.Generator(device=dev()).manual_seed(1)
    want = p0.clone()
    for k in range(2):
        held = step.slot.clone()
        step.step([torch.randn(S, generator=g, device=dev())])
        assert torch.equal(step.master[rest], p0[rest]) and torch.equal(step.slot[rest], held[rest])
        want = torch.from_numpy(R.update(want.cpu().numpy(), step.o_shard.float().cpu().numpy(), 0.1, 0.1)).to(dev())
        assert torch.equal(step.master[inside], want[inside])
        assert torch.equal(step.slot.view(BF)[inside], want.to(BF)[inside])
        # another optimizer's step
        step.slot[rest] = 77 + k
    # resumed: a slot that others write too keeps what is theirs
    other = torch.full((S,), 5, dtype=torch.int16, device=dev()) if given else None
    again = new(Z, S, matrices=mats, weight_decay=0.1, slot=other)
    if given:
        other[rest] = 9
    again.load_state_dict(step.state_dict())
    assert torch.equal(again.slot.view(BF)[inside], want.to(BF)[inside])
    assert bool((again.slot[rest] == 9).all()) if given else torch.equal(again.slot.view(BF), again.master.to(BF))
    assert torch.equal(again.master, step.master) and torch.equal(again.m, step.m)


def test_strides_of_a_stack(Z):
    """Rows and matrices further apart than they need be; and what the documentation excludes,
    matrices between another's rows, refused for x as for out."""
    g = torch.Generator(device=dev()).manual_seed(2)
    both = torch.randn(6, 40, 90, generator=g, device=dev())
    x = both[::2, 4:30, 8:60]
    want = Z.zero_orthogonalize(x.contiguous())
    assert torch.equal(Z.zero_orthogonalize(x), want)
    out = torch.zeros(6, 40, 90, dtype=BF, device=dev())
    assert torch.equal(Z.zero_orthogonalize(x, out=out[1::2, :26, :52]), want)
    assert bool((out[::2] == 0).all())
    heads = torch.randn(26, 3 * 52, generator=g, device=dev()).view(26, 3, 52).transpose(0, 1)
    for kw in (dict(x=heads), dict(x=x, out=torch.zeros(26, 3, 52, dtype=BF, device=dev()).transpose(0, 1))):
        with pytest.raises(Z.ZeroError, match="batch stride"):
            Z.zero_orthogonalize(**kw)
    with pytest.raises(Z.ZeroError, match="column stride"):
        Z.zero_orthogonalize(x.transpose(1, 2))


def test_a_shard_without_matrices(Z):
    """Its matrices lie in other shards: it folds, counts and agrees as they do, and writes nothing."""
    step = new(Z, 96, matrices=[(0, 8, 8), (4000, 8, 8)], shard_off=200, weight_decay=0.1)
    was, slot = step.master.clone(), step.slot.clone()
    st, verdict = step.step([torch.ones(96, device=dev())])
    assert verdict == Z.ZERO_COMMIT and step.t == 1 and st.sumsq == 96.0
    assert step.runs == [] and torch.equal(step.master, was) and torch.equal(step.slot, slot)
    st, verdict = step.step([torch.full((96,), float("inf"), device=dev())])
    assert verdict == Z.ZERO_SKIP and step.t == 1
