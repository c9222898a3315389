"""MuonShardStep's refusals that need no GPU."""
import pytest
import torch

import zero_partitioned_optimizer_amd as Z


@pytest.mark.parametrize("bad,word", [
    (dict(lr=-0.1), "lr="), (dict(weight_decay=float("nan")), "weight_decay="), (dict(mu=1.0), "mu="),
    (dict(steps=0), "steps=0"), (dict(steps=65), "steps=65"), (dict(steps=9), "multiply to"), (dict(eps=0.0), "eps="),
    (dict(coefficients=(1.0, 2.0)), "neither three numbers"), (dict(coefficients=(float("inf"), 0.0, 0.0)), "coefficient"),
    (dict(scale=lambda r, c: 1e5), "scale="), (dict(matrices=[(0, 1 << 16, 1 << 16)]), "smaller side"),
    (dict(matrices=[(0, 1, (1 << 20) + 1)]), "larger")], ids=str)
def test_bad_values_are_refused_by_the_constructor(bad, word):
    """Not by the last part of a step, which would leave it half done."""
    kw = {"lr": 0.1, "matrices": [(0, 5, 10)], **bad}
    with pytest.raises(Z.ZeroError, match=word):
        Z.MuonShardStep(100, 1, Z.ZERO_F32, torch.zeros(100), kw.pop("matrices"), **kw)


def test_runs_that_an_update_writes():
    """The shard's part of the matrices and of gaps shorter than the padding behind them."""
    runs = Z.MuonShardStep._runs
    spans = [(0, 100), (100, 50), (158, 42), (300, 100), (410, 90)]
    assert runs(spans, 0, 520, 16) == [(0, 200), (300, 500)]
    assert runs(spans, 0, 515, 16) == [(0, 200), (300, 515)]            # the shard ends 15 behind the last
    assert runs(spans, 0, 515, 0) == [(0, 150), (158, 200), (300, 400), (410, 500)]
    assert runs(spans, 0, 515, 9) == [(0, 200), (300, 400), (410, 500)]
    # cut by the shard, within a matrix, a gap that is padding and one that is not
    assert runs(spans, 120, 35, 16) == [(0, 35)] and runs(spans, 152, 100, 16) == [(0, 48)]
    assert runs(spans, 200, 100, 16) == [] and runs(spans, 210, 100, 16) == [(90, 100)]
    # a short shard that holds no matrix
    assert runs(spans, 505, 10, 16) == [] and runs([], 0, 8, 16) == []
