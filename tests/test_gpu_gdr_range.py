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


# ------------------------------------------------------------------ bf16 token by token
TOKENWISE = [(1, 4, 2, 16, 64, 64), (1, 1, 1, 1, 128, 128), (2, 2, 1, 31, 128, 128), (2, 2, 2, 63, 64, 128),
             (1, 2, 1, 64, 128, 64), (1, 2, 2, 127, 128, 128), (1, 2, 1, 128, 128, 128), (1, 2, 1, 240, 128, 128),
             (1, 2, 1, 300, 64, 64), (1, 2, 2, 700, 32, 16), (2, 4, 1, 333, 16, 128)]


@pytest.mark.parametrize("Bn,H,Hk,T,dk,dv", TOKENWISE)
def test_bf16_outputs_of_float32_arithmetic(B, monkeypatch, Bn, H, Hk, T, dk, dv):
    """Token by token a bf16 output is a float32 value rounded once, at every head size."""
    monkeypatch.setattr(base, "tol_out", lambda x: 2.0 ** -8 + TOL_F32)
    x = draw(Bn, H, Hk, T, dk, dv, seed=50)
    fwd, bwd = launches(B, x)
    assert fwd == 1
    check_fwd(B, x)
    if bwd == 2:
        check_bwd(B, x)


def test_the_same_call_twice(B):
    """Nothing in a call depends on the order in which its blocks run."""
    for starts in (None, [0, 130, 131, 700, 900]):
        x = draw(1, 16, 8, 900, 128, 128, n=4 if starts else None, seed=51)
        f, g = gpu_fwd(B, x, starts), gpu_bwd(B, x, starts)
        for _ in range(3):
            assert all(np.array_equal(a, b) for a, b in zip(gpu_fwd(B, x, starts), f))
            assert all(np.array_equal(a, b) for a, b in zip(gpu_bwd(B, x, starts), g))
