"""The gated delta rule over the whole range that its declaration allows: keys and
gates that let states, written rows and their products grow, key lengths that
differ, long memories, gates at zero, and bad values in the middle of a sequence.
Against the recurrence in 64 bits; tolerances as in test_gpu_gdr.py."""

import numpy as np
import pytest
import torch

from oracle import gdr
from tests import test_gpu_gdr as base
from tests._parity import TOL_F32, rel_err
from tests.test_gpu_gdr import B, DEV, check_bwd, check_fwd, draw, gpu_bwd, gpu_fwd, launches  # noqa: F401

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "log_alpha", "beta")


# ------------------------------------------------------------------ written rows
@pytest.mark.parametrize("shift", [4, 8])
def test_short_keys_with_large_gates(B, shift):
    """Keys of length 2^-shift, beta |k|^2 below 1 as before: beta v is 2^(2 shift) times v."""
    x = draw(1, 2, 1, 520, 128, 128, seed=42)
    x["k"] = x["k"] * 2.0 ** -shift
    x["beta"] = x["beta"] * 4.0 ** shift
    assert launches(B, x) == (3, 4)
    check_fwd(B, x)
    check_bwd(B, x)


# ------------------------------------------------------------------ the inverse
@pytest.mark.parametrize("ratio", [2.0 ** 6, 2.0 ** 11])
def test_key_lengths_that_differ(B, ratio):
    """Nearly parallel keys, every 16 in turn short and long, beta |k|^2 = 1 throughout: what a
    long key reads of the rows that short ones wrote is `ratio` times these rows' values."""
    T = 400
    x = draw(1, 2, 1, T, 128, 128, seed=43)
    k = torch.nn.functional.normalize(torch.ones(128) + 0.5 * x["k"].float() * 128 ** 0.5, dim=-1)
    long = ((torch.arange(T) // 16) % 2).view(1, 1, T, 1)
    x["k"] = (k * torch.where(long == 1, ratio ** 0.5, ratio ** -0.5)).to(torch.bfloat16)
    x["beta"] = (1.0 / x["k"].double().square().sum(-1)).float().expand(1, 2, T).contiguous()
    assert launches(B, x) == (3, 4)
    check_fwd(B, x)
    check_bwd(B, x)
