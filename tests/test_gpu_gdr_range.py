"""The gated delta rule over the whole range that its declaration allows: keys and
gates that let states, written rows and their products grow, key lengths that
differ, long memories, gates at zero, and bad values in the middle of a sequence.
Against the recurrence in 64 bits; tolerances as in test_gpu_gdr.py."""

import numpy as np
import pytest
import torch

from oracle import gdr
from tests import test_gpu_gdr as base
from tests._parity import TOL_BF16, TOL_F32, rel_err
from tests.test_gpu_gdr import B, DEV, check_bwd, check_fwd, draw, gpu_bwd, gpu_fwd, launches  # noqa: F401

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "log_alpha", "beta")


# ------------------------------------------------------------------ products of the gradient
def repeated(n):
    """Tolerance of states and gates' gradients where n tokens (of a chunk) have one key and beta |k|^2
    up to 2.  Their rows e solve (I + A diag(beta)) e = ..., whose entries and whose inverse's are 2 at
    most: 2 n to a row.  The computed ones solve it up to 2^-21 of its terms (operands in two fp16 parts,
    3 x 2^-24 each product, and its sum), so that they are off by 2^-21 (2 n) (2 n) of the largest."""
    return 2.0 ** -21 * (2 * n) ** 2


def terms_of_dk(x, scale):
    """The largest sum of magnitudes that make up an element of dk, over the largest |dk|, for sequences
    of one chunk without decay: R^T Q, u D, (N + N^T) K and (beta w) S, N = (beta w) u^T below the diagonal."""
    terms, dk = 0.0, 0.0
    for _, (q, k, v, la, b), do, S, D in base.slices(x, None):
        dk = dk + gdr.backward(q, k, v, la, b, do, scale=scale, state=S, dstate=D)["dk"]
        S0, D1, u, w = np.abs(S), np.abs(D), np.zeros_like(v), np.zeros_like(v)
        for t in range(len(q)):
            u[t] = b[t] * (v[t] - S @ k[t])
            S = S + np.outer(u[t], k[t])
        for t in reversed(range(len(q))):
            D = D + scale * np.outer(do[t], q[t])
            w[t] = b[t] * D @ k[t]
            D = D - np.outer(w[t], k[t])
        u, w = np.abs(u), np.abs(w)
        N, R = np.tril(w @ u.T, -1), np.tril(scale * np.abs(do) @ u.T)
        terms = terms + R.T @ np.abs(q) + u @ D1 + (N + N.T) @ np.abs(k) + w @ S0
    return terms.max() / np.abs(dk).max()


def flat_key(T, d, length):
    """One key of equal elements at every token."""
    return torch.full((1, 1, T, d), length / d ** 0.5, dtype=torch.bfloat16)


@pytest.mark.parametrize("T", [64, 512])
def test_gradient_of_repeated_keys(B, monkeypatch, T):
    """beta |k|^2 just below 2, one key throughout and values of alternating sign: at 512 tokens the
    state grows 71-fold and the written rows 1600-fold over the largest value."""
    x = draw(1, 1, 1, T, 128, 128, seed=40)
    x["k"] = flat_key(T, 128, 1.0)
    x["beta"][:] = 1.999
    x["log_alpha"][:] = 0.0
    x["v"] = (1.0 - 2.0 * (torch.arange(T) % 2)).view(1, 1, T, 1).expand(1, 1, T, 128).contiguous().to(torch.bfloat16)
    x["dout"] = torch.ones_like(x["v"])
    del x["state_in"], x["dstate_out"]
    assert launches(B, x)[1] == 4
    monkeypatch.setattr(base, "TOL_F32", repeated(min(T, 128)))
    check_fwd(B, x)
    check_bwd(B, x)


@pytest.mark.parametrize("sq", [1.0, 1.89])
def test_gradient_of_constant_states(B, monkeypatch, sq):
    """Flat states and adjoints that do not grow, flat keys with beta |k|^2 up to 1.89: a written row is
    11 times any element of the state, and so is a row of w."""
    x = draw(1, 2, 1, 64, 128, 128, seed=41)
    x["k"] = flat_key(64, 128, sq ** 0.5)
    x["beta"][:] = 2.0 if sq == 1.0 else 1.0
    x["log_alpha"][:] = 0.0
    x["state_in"][:] = 1.9
    x["dstate_out"][:] = 1.9
    assert launches(B, x)[1] == 4
    monkeypatch.setattr(base, "TOL_F32", repeated(64))
    check_fwd(B, x)
    # dk is a sum of terms that cancel: operands of one fp16 part, half a step (2^-11) each, three of them in N's
    # terms (its two factors and itself), two in the others
    terms = terms_of_dk(x, 0.5)
    monkeypatch.setattr(base, "tol_out", lambda x: max(TOL_BF16, 2.0 ** -8 + 3 * 2.0 ** -11 * terms))
    check_bwd(B, x)


def test_gradient_of_aligned_rows(B):
    """The shortest keys, all one, and values of alternating sign: the rows u that every token writes
    are 4096 in the scale of the operands, and with dout constant their product adds up over d_v:
    128 x 15.5 x 3928."""
    T = 300
    x = draw(1, 2, 1, T, 128, 128, seed=57, init=False)
    x["k"] = flat_key(T, 128, 2.0 ** -12)
    x["beta"][:] = 0.99 * 4.0 ** 12
    x["log_alpha"][:] = 0.0
    sign = (1.0 - 2.0 * (torch.arange(T) % 2)).view(1, 1, T, 1)
    x["v"] = (1.9375 * sign).expand(1, 2, T, 128).contiguous().to(torch.bfloat16)
    x["dout"] = torch.full_like(x["dout"], 1.9375)
    assert launches(B, x) == (3, 4)
    check_fwd(B, x)
    got = gpu_bwd(B, x)
    ref = [np.zeros(got[0].shape), np.zeros(got[1].shape)]
    for _, a, do, _, _ in base.slices(x, None):
        r = gdr.backward(*a, do, scale=0.5)
        ref[0][0, 0] += r["dq"]
        ref[1][0, 0] += r["dk"]
    assert all(rel_err(y, z, 1) <= TOL_BF16 for y, z in zip(got, ref)) and all(np.isfinite(y).all() for y in got)


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


@pytest.mark.parametrize("shift", [6, 12])
def test_long_keys_with_small_gates(B, shift):
    """Keys of length 2^shift, beta |k|^2 below 1 as before."""
    x = draw(1, 2, 1, 520, 128, 128, seed=54)
    x["k"] = x["k"] * 2.0 ** shift
    x["beta"] = x["beta"] * 4.0 ** -shift
    assert launches(B, x) == (3, 4)
    check_fwd(B, x)
    check_bwd(B, x)


@pytest.mark.parametrize("k", [-90, 120])
def test_values_at_the_ends_of_float(B, k):
    """Values and states scaled by 2^k scale the outputs by it (as test_scaling_by_powers_of_two_is_exact,
    further out): an intermediate of their size times that of a key's inverse length must not overflow."""
    x = draw(2, 4, 2, 300, 128, 128, seed=55)
    y = {n: t * 2.0 ** k if n in ("v", "state_in") else t for n, t in x.items()}
    for a, b in zip(gpu_fwd(B, x), gpu_fwd(B, y)):
        assert np.array_equal(b, a * np.float32(2.0 ** k))


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


# ------------------------------------------------------------------ long memories
@pytest.mark.parametrize("d,io,T", [(32, "f32", 4000), (128, "f32", 1500), (16, "bf16", 4000), (64, "bf16", 250)])
def test_decay_near_one_token_by_token(B, d, io, T):
    """alpha = 0.9999 and faint writes: a state is scaled by thousands of decays, whose
    roundings must not lean to one side."""
    x = draw(1, 2, 1, T, d, d, io, seed=44)
    x["log_alpha"][:] = -1e-4
    x["beta"] *= 0.02
    assert launches(B, x)[0] == 1
    check_fwd(B, x)
    if launches(B, x)[1] == 2:
        check_bwd(B, x)


@pytest.mark.parametrize("la", [-1.3e-6, -1e-4])
@pytest.mark.parametrize("d,io,T", [(64, "bf16", 131072), (32, "f32", 131072)])
def test_long_memories(B, d, io, T, la):
    """Nothing is written: a state and its adjoint are what T decays leave of them.  Token by token a float32
    state itself is rounded T times, by up to 2^-24 each; as it moves by the same few steps a token, to the
    same side for long."""
    g = torch.Generator(device=DEV).manual_seed(52)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    q, k, v = (torch.nn.functional.normalize(torch.randn(1, 1, T, d, generator=g, device=DEV), dim=-1).to(dt) for _ in range(3))
    gate, zero = torch.full((1, 1, T), la, device=DEV), torch.zeros(1, 1, T, device=DEV)
    s, ds = (torch.randn(1, 1, d, d, generator=g, device=DEV) for _ in range(2))
    left = np.exp(T * np.float64(np.float32(la)))
    out, tol = torch.empty_like(s), TOL_F32 if io == "bf16" else TOL_F32 + T * 2.0 ** -24
    B.ll_gdr_fwd(q, k, v, gate, zero, state_in=s, state_out=out)
    err = rel_err(out.cpu().numpy(), s.double().cpu().numpy() * left, 0)
    assert err <= tol
    B.ll_gdr_bwd(q, k, v, gate, zero, torch.zeros_like(v), state_in=s, dstate_out=ds, dstate_in=out)
    assert B.ll_last_device_error() == 0
    err = rel_err(out.cpu().numpy(), ds.double().cpu().numpy() * left, 0)
    assert err <= tol


@pytest.mark.parametrize("la", [-1e-4, -0.37, -0.53, -3.0, -90.0, -float("inf")])
def test_constant_decays_token_by_token(B, la):
    x = draw(1, 2, 1, 300, 32, 32, "f32", seed=45)
    x["log_alpha"][:] = la
    check_fwd(B, x)
    check_bwd(B, x)


def test_decay_near_one_in_decode_steps(B):
    T, H, d = 3000, 2, 32
    x = draw(1, H, 1, T, d, d, "f32", seed=46)
    x["log_alpha"][:] = -1e-4
    x["beta"] *= 0.02
    g = {n: x[n].to(DEV) for n in NAMES}
    st = x["state_in"].to(DEV)
    steps = [g[n].transpose(1, 2).transpose(0, 1).contiguous() for n in NAMES]  # [T, 1, heads, ...]
    for t in range(T):
        B.ll_gdr_decode_step(*[s[t] for s in steps[:3]], steps[3][t].clone(), steps[4][t].clone(), st)
    assert B.ll_last_device_error() == 0
    for (i, b, h, hk, lo, hi), a, _, s0, _ in base.slices(x, None):
        assert rel_err(st[i, h].cpu().numpy(), gdr.forward(*a, state=s0)[1], 0) <= TOL_F32


# ------------------------------------------------------------------ alpha = 0
@pytest.mark.parametrize("d,io,T", [(128, "bf16", 700), (64, "f32", 300), (32, "bf16", 200)])
@pytest.mark.parametrize("la", [-float("inf"), -200.0])
def test_no_gradient_by_a_decay_of_zero(B, d, io, T, la):
    """alpha = 0 in float32: what came before does not matter, and neither does alpha's logarithm."""
    x = draw(1, 2, 1, T, d, d, io, seed=47)
    at = [0, 1, 50, 127, 128, T - 1]
    x["log_alpha"][:, :, at] = la
    got = gpu_bwd(B, x)[3]
    assert (got[:, :, at] == 0.0).all()
    assert (got != 0.0).sum() > got.size // 2


# ------------------------------------------------------------------ bad values inside a sequence
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d,io,T,at,first", [(128, "bf16", 700, 300, 256), (64, "bf16", 600, 390, 384),
                                             (128, "f32", 100, 37, 37), (128, "bf16", 60, 37, 37)])
def test_a_bad_value_leaves_what_is_before_it(B, d, io, T, at, first, bad):
    """In chunks: whole chunks before the bad token's; token by token: every token before it."""
    x = draw(1, 2, 1, T, d, d, io, seed=48)
    x["v"][:, 0, at, 3] = 0.0
    ref = gpu_fwd(B, x)[0]
    x["v"][:, 0, at, 3] = bad
    o, s = gpu_fwd(B, x)
    assert np.array_equal(o[:, 0, :first], ref[:, 0, :first]) and np.array_equal(o[:, 1], ref[:, 1])
    assert not np.isfinite(o[0, 0, at, 3]) and not np.isfinite(s[0, 0, 3]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["q", "k", "log_alpha", "beta"])
@pytest.mark.parametrize("d,io,T,at,first", [(128, "bf16", 700, 300, 256), (128, "f32", 100, 37, 37)])
def test_a_bad_key_or_gate_leaves_what_is_before_it(B, d, io, T, at, first, name, bad):
    x = draw(1, 2, 1, T, d, d, io, seed=53)
    x[name][(0, 0, at, 3) if name in "qk" else (0, 0, at)] = 0.0
    ref = gpu_fwd(B, x)[0]
    x[name][(0, 0, at, 3) if name in "qk" else (0, 0, at)] = bad
    o = gpu_fwd(B, x)[0]
    assert np.array_equal(o[:, :, :first], ref[:, :, :first]) and not np.isfinite(o[0, 0, at]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("d,io,T,at", [(128, "bf16", 700, 300), (64, "f32", 200, 70)])
def test_gradients_beside_a_bad_value(B, d, io, T, at, bad):
    """A bad v reaches no chunk before its own, a bad dout none behind it."""
    C = 128 if io == "bf16" else 64
    x = draw(1, 2, 1, T, d, d, io, seed=49)
    x["v"][:, 0, at, 3] = 0.0
    x["dout"][:, 0, at, 3] = 0.0
    ref = gpu_bwd(B, x)
    before, behind = at // C * C, (at // C + 1) * C
    y = {n: t.clone() for n, t in x.items()}
    y["v"][:, 0, at, 3] = bad
    got = gpu_bwd(B, y)
    for a, b in zip(got[:5], ref[:5]):
        assert np.array_equal(a[:, 0, :before], b[:, 0, :before])
    for a, b in zip(got[2:5], ref[2:5]):
        assert np.array_equal(a[:, 1], b[:, 1])
    y = {n: t.clone() for n, t in x.items()}
    y["dout"][:, 0, at, 3] = bad
    got = gpu_bwd(B, y)
    for a, b in zip(got[:5], ref[:5]):
        assert np.array_equal(a[:, 0, behind:], b[:, 0, behind:])
    for a, b in zip(got[2:5], ref[2:5]):
        assert np.array_equal(a[:, 1], b[:, 1])


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


# ------------------------------------------------------------------ a slot handed on
@pytest.mark.parametrize("io,d", [("bf16", 128), ("f32", 32)])
def test_decode_forgets_whatever_a_slot_holds(B, io, d):
    H = 2
    x = {n: t.to(DEV) for n, t in draw(3, H, 1, 1, d, d, io, seed=56).items()}
    args = [x[n][:, :, 0].contiguous() for n in NAMES]
    args[3][1] = -float("inf")
    states = torch.randn(3, H, d, d, device=DEV)
    clean = states.clone()
    clean[1] = 0.0
    want = B.ll_gdr_decode_step(*args, clean)
    states[1, 0, :, ::3], states[1, 1] = float("nan"), float("inf")
    o = B.ll_gdr_decode_step(*args, states)
    assert torch.equal(o, want) and torch.equal(states, clean) and B.ll_last_device_error() == 0
