"""The combination cases' positions (perf/more_operators.py), made on the CPU: every place that is not dropped names a
row that is there, and no row twice.  A position past the rows would have the plain form read out of range."""

import pytest
import torch
from torch.overrides import TorchFunctionMode

from perf import more_operators


class _OnHost(TorchFunctionMode):
    def __torch_function__(self, func, types, args=(), kwargs=None):
        kwargs = dict(kwargs or {})
        if kwargs.get("device") == "cuda":
            kwargs["device"] = "cpu"
        return func(*args, **kwargs)


@pytest.mark.parametrize("drop", [0.0, 0.4, 0.5])
@pytest.mark.parametrize("k", [1, 2, 3, 8, 10])
def test_positions_name_rows_that_are_there(k, drop):
    for T in (1, 2, 3, 7, 8, 15, 16, 17, 40):
        for seed in range(40):
            with _OnHost():
                positions, R = more_operators._plan(torch.Generator().manual_seed(seed), T, k, drop)
            kept = positions[positions >= 0]
            assert R == T * k - int(drop * T * k) and positions.shape == (T, k)
            assert torch.equal(kept.sort()[0], torch.arange(R, dtype=torch.int32)), (T, seed, positions, R)
