"""The surrounding operators at the ends of their ranges: moments that are not numbers."""
import numpy as np
import pytest
import torch

from residual_binarized_weight_b200 import rbw
from tests.test_adamw_gpu import F32, make, reference, upload

gpu = pytest.mark.gpu
DEV = "cuda"


# ---------------------------------------------------------------- optimizer
@gpu
@pytest.mark.parametrize("n,at", [(600, 300), (256, 0), (700, 699)])
def test_a_second_moment_of_nan_stays(n, at):
    """8-bit states: NaN in a gradient is NaN in both moments, in this step and the next; the other elements of the
    block are as if that element were 0 (its moments start from 0), bit for bit."""
    t = make(n, 8, F32, F32, 6)
    for name in ("m", "v"):
        t[name].view(torch.uint8)[at] = 0
    t["g"][at] = 0
    want = reference(t, 3, 0, 11)
    t["g"][at] = np.nan
    T = upload(t)
    opt = rbw.AdamW([T], seed=11)
    opt.step(3)
    others = torch.arange(n) != at
    for got, name in ((T.exp_avg, "m"), (T.exp_avg_sq, "v")):
        assert bool(torch.isnan(got.float())[at]), name
        assert torch.equal(got.cpu().view(torch.uint8)[others], want[name].view(torch.uint8)[others]), name
    for got, name in ((T.exp_avg_scale, "ms"), (T.exp_avg_sq_scale, "vs")):
        assert np.array_equal(got.cpu().numpy(), want[name]), name
    T.grad.nan_to_num_(0.0)
    opt.step(4)
    for got in (T.exp_avg, T.exp_avg_sq, T.param):
        assert int(torch.isnan(got.float()).sum()) == 1 and bool(torch.isnan(got.float())[at])
