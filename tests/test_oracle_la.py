"""The float64 oracle of linear attention with a decay per head against other
forms of the same mathematics, and the host side of its entry points (CPU)."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import la, mamba2

RNG = np.random.default_rng


def draw(T, dk, dv, seed=0):
    r = RNG(seed)
    return (r.standard_normal((T, dk)), r.standard_normal((T, dk)), r.standard_normal((T, dv)),
            -0.3 * r.random(T), r.standard_normal((T, dv)), r.standard_normal((dv, dk)), r.standard_normal((dv, dk)))


def test_forward_is_the_masked_product():
    q, k, v, g, _, s0, _ = draw(23, 8, 5)
    o, s = la.forward(q, k, v, g, 0.7, s0)
    c = np.cumsum(g)
    m = np.tril(np.exp(c[:, None] - c[None, :]))
    assert np.allclose(o, 0.7 * ((q @ k.T * m) @ v + np.exp(c)[:, None] * (q @ s0.T)), atol=1e-12)
    assert np.allclose(s, np.exp(c[-1]) * s0 + (v * np.exp(c[-1] - c)[:, None]).T @ k, atol=1e-12)


def test_forward_is_the_log_linear_one_with_every_lambda_one():
    q, k, v, g, _, _, _ = draw(33, 16, 16, 3)
    o, _ = la.forward(q, k, v, g)
    ref = mamba2.forward_dense_bh(*[x[None, None] for x in (q, k, v, g)], np.ones((1, 1, 33, 7)))[0, 0]
    assert np.allclose(o, ref, atol=1e-10)


def test_backward_against_differences():
    q, k, v, g, do, s0, ds = draw(7, 4, 3, 1)
    grads = la.backward(q, k, v, g, do, 0.6, s0, ds)

    def f(*a):
        o, s = la.forward(*a[:4], 0.6, a[4])
        return np.sum(o * do) + np.sum(s * ds)

    args = [q, k, v, g, s0]
    for n, name in enumerate(("dq", "dk", "dv", "dlog_alpha", "dstate_in")):
        for at in np.ndindex(args[n].shape):
            hi, lo = [x.copy() for x in args], [x.copy() for x in args]
            hi[n][at] += 1e-6
            lo[n][at] -= 1e-6
            assert abs((f(*hi) - f(*lo)) / 2e-6 - grads[name][at]) < 1e-7, (name, at)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_against_its_formula_and_transpose(inter):
    r = RNG(5)
    x, y, f = r.standard_normal((3, 9, 16)), r.standard_normal((3, 9, 16)), 10000.0 ** (-np.arange(5) / 5)
    pos = np.arange(9) * 7 - 20
    got = la.rope(x, pos, f, inter, 1.3)
    want = x.copy()
    for i in range(5):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + 5)
        c, s = np.cos(pos * f[i]), np.sin(pos * f[i])
        want[..., a], want[..., b] = 1.3 * (x[..., a] * c - x[..., b] * s), 1.3 * (x[..., a] * s + x[..., b] * c)
    assert np.allclose(got, want, atol=1e-12)
    assert np.isclose((got * y).sum(), (x * la.rope(y, pos, f, inter, 1.3, back=True)).sum())


def test_rope_scores_depend_on_distance_alone():
    r = RNG(6)
    q, k, f = r.standard_normal((1, 8)), r.standard_normal((1, 8)), 100.0 ** (-np.arange(4) / 4)
    a = la.rope(q, [1000005], f) @ la.rope(k, [1000000], f).T
    assert np.allclose(a, la.rope(q, [5], f) @ la.rope(k, [0], f).T, atol=1e-9)


# ---------------------------------------------------------------- the host side of the entry points
FAKE = 0x7f0000000000  # never dereferenced: every case below fails a host-side check first


@pytest.fixture(scope="module")
def B():
    import os
    from log_linear_attention_chunked_gb300 import binding
    if not os.path.exists(binding.LIB_PATH):
        from log_linear_attention_chunked_gb300 import build
        build.build()
    binding.lib()
    return binding


def _shape(binding, **kw):
    d = dict(B=1, H=4, Hk=2, T=64, dk=64, dv=64, n_seqs=0, scale=1.0, io=binding.LL_BF16, per_head=False)
    d.update(kw)
    return binding.make_la_shape(**d)


BAD_SHAPES = [(dict(B=0), 1), (dict(T=0), 1), (dict(Hk=3), 1), (dict(Hk=0), 1), (dict(io=2), 1), (dict(dk=96), 2),
              (dict(dv=256), 2), (dict(n_seqs=-1), 1), (dict(n_seqs=2, B=2), 1), (dict(scale=math.inf), 1),
              (dict(scale=math.nan), 1), (dict(T=0x7fffffff - 512), 2), (dict(B=1 << 20, T=4096, H=64, Hk=64), 2)]


def _call(B, name, shape, ptrs, starts=None, ws=FAKE + (60 << 32), ws_bytes=1 << 50):
    vp = ctypes.c_void_p
    return getattr(B.lib(), name)(ctypes.byref(shape), vp(starts) if starts else None,
                                  *[vp(x) if x else None for x in ptrs], vp(ws) if ws else None, ws_bytes, None)


@pytest.mark.parametrize("name,count,need,outs", [
    ("ll_la_fwd", 7, (0, 1, 2, 3, 5), (5, 6)),                        # q k v la state_in | o state_out
    ("ll_la_bwd", 12, (0, 1, 2, 3, 5, 7, 8, 9, 10), (7, 8, 9, 10, 11))])  # q k v la state_in dout dstate_out | ...
def test_sequences_refuse_bad_arguments_on_the_host(B, name, count, need, outs):
    good = [FAKE + (i << 32) for i in range(count)]
    for kw, code in BAD_SHAPES:
        assert _call(B, name, _shape(B, **kw), good) == code, kw
        assert getattr(B, name + "_workspace_size")(_shape(B, **kw)) == 0
        assert getattr(B, name + "_launches")(_shape(B, **kw)) == 0
    ok = _shape(B, T=4096)
    assert getattr(B, name + "_launches")(ok) >= 1
    need_ws = getattr(B, name + "_workspace_size")(ok)
    assert need_ws > 0
    for i in need:
        assert _call(B, name, ok, [0 if j == i else p for j, p in enumerate(good)]) == 1, i
    for i in range(count):
        assert _call(B, name, ok, [p + (4 if j == i else 0) for j, p in enumerate(good)]) == 1, i
    for i in outs:           # every output on every other tensor, but the state that may be updated in place
        for j in range(count):
            if i == j or (name, i, j) in (("ll_la_fwd", 6, 4), ("ll_la_bwd", 11, 6)):
                continue
            assert _call(B, name, ok, [good[j] + 16 if n == i else p for n, p in enumerate(good)]) == 1, (i, j)
    assert _call(B, name, ok, good, starts=FAKE + (50 << 32)) == 1           # starts without sequences
    assert _call(B, name, _shape(B, n_seqs=3), good) == 1                    # and the other way round
    assert _call(B, name, ok, good, ws=0) == 5
    assert _call(B, name, ok, good, ws_bytes=need_ws - 1) == 5
    assert _call(B, name, ok, good, ws=FAKE + (60 << 32) + 128) == 5
    odd = _shape(B, T=4096)
    odd.per_head = 2
    assert _call(B, name, odd, good) == 1


def test_step_refuses_bad_arguments_on_the_host(B):
    vp = ctypes.c_void_p
    rope = B.ll_rope(64, 0, 1.0, FAKE + (30 << 32))

    def call(dims=(2, 4, 2, 64, 64), io=1, per_head=0, scale=1.0, slots=FAKE + (20 << 32), n=4, r=rope, pos=FAKE + (21 << 32), ptrs=None):
        p = ptrs or [FAKE + (i << 32) for i in range(6)]
        return B.lib().ll_la_decode_step(*dims, io, per_head, scale, vp(slots) if slots else None, n,
                                         ctypes.byref(r) if r else None, vp(pos) if pos else None,
                                         *[vp(x) if x else None for x in p], None)

    for dims, code in (((0, 4, 2, 64, 64), 1), ((2, 4, 3, 64, 64), 1), ((2, 4, 2, 48, 64), 2), ((2, 4, 2, 64, 256), 2),
                       ((1 << 22, 64, 2, 64, 64), 2)):
        assert call(dims) == code, dims
    assert call(io=3) == 1 and call(per_head=2) == 1 and call(scale=math.nan) == 1 and call(n=0) == 1
    assert call(slots=0, n=1) == 1
    assert call(r=None) == 1 and call(pos=0) == 1                            # one without the other
    for bad in (B.ll_rope(0, 0, 1.0, FAKE), B.ll_rope(63, 0, 1.0, FAKE), B.ll_rope(66, 0, 1.0, FAKE),
                B.ll_rope(64, 2, 1.0, FAKE), B.ll_rope(64, 0, math.inf, FAKE), B.ll_rope(64, 0, 1.0, None),
                B.ll_rope(64, 0, 1.0, FAKE + 4)):
        assert call(r=bad) == 1
    good = [FAKE + (i << 32) for i in range(6)]
    for i in range(6):
        assert call(ptrs=[0 if j == i else p for j, p in enumerate(good)]) == 1
        assert call(ptrs=[p + (8 if j == i else 0) for j, p in enumerate(good)]) == 1
    assert call(ptrs=good[:5] + [good[2]]) == 1                              # o on v
    assert call(ptrs=good[:5] + [good[4] + 64]) == 1                         # o in the states
    assert call(slots=good[4] + 16) == 1                                     # slots in the states
    assert call(r=B.ll_rope(64, 0, 1.0, good[5])) == 1                       # frequencies on o


def test_rope_refuses_bad_arguments_on_the_host(B):
    vp = ctypes.c_void_p
    good = [FAKE + (i << 32) for i in range(4)]

    def call(dims=(2, 4, 2, 5, 64), io=0, r=B.ll_rope(64, 0, 1.0, FAKE + (30 << 32)), pos=FAKE + (21 << 32), ptrs=good, name="ll_rope_fwd"):
        return getattr(B.lib(), name)(*dims, io, ctypes.byref(r) if r else None, vp(pos) if pos else None,
                                      *[vp(x) if x else None for x in ptrs], None)

    for name in ("ll_rope_fwd", "ll_rope_bwd"):
        for dims, code in (((0, 4, 2, 5, 64), 1), ((2, 0, 2, 5, 64), 1), ((2, 4, 0, 5, 64), 1), ((2, 4, 2, 0, 64), 1),
                           ((2, 4, 2, 5, 80), 2), ((1 << 20, 4, 2, 1 << 12, 64), 2), ((1, 60000, 6000, 5, 64), 2)):
            assert call(dims, name=name) == code, dims
        assert call(r=None, name=name) == 1 and call(io=7, name=name) == 1
        assert call(r=B.ll_rope(66, 0, 1.0, FAKE), name=name) == 1 and call(r=B.ll_rope(7, 0, 1.0, FAKE), name=name) == 1
        assert call(r=B.ll_rope(64, 0, math.nan, FAKE), name=name) == 1
        assert call(ptrs=[0, good[1], good[2], good[3]], name=name) == 1
        assert call(ptrs=[good[0], 0, good[2], good[3]], name=name) == 1     # k_out without k
        assert call(ptrs=[good[0], good[1], good[2], 0], name=name) == 1
        assert call(ptrs=[good[0], good[1], good[0] + 16, good[3]], name=name) == 1   # shifted in place
        assert call(ptrs=[good[0], good[1], good[1], good[3]], name=name) == 1        # q_out on k
        assert call(ptrs=[good[0], good[1], good[2], good[2]], name=name) == 1        # both outputs in one place
        assert call(pos=good[2] + 16, name=name) == 1
        assert call(pos=FAKE + (21 << 32) + 8, name=name) == 1


def test_frequencies(B):
    f = B.ll_rope_freqs(64, 10000.0).double()
    plain = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    assert torch.allclose(f, plain, rtol=2 ** -23, atol=0)
    assert torch.allclose(B.ll_rope_freqs(64, 10000.0, factor=4.0).double(), plain / 4, rtol=2 ** -23, atol=0)
    got = B.ll_rope_freqs(128, 10000.0, factor=16.0, length=4096.0).double()
    base = 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)
    turns = 4096 * base / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    assert torch.allclose(got, base * keep + base / 16 * (1 - keep), rtol=2 ** -23, atol=0)
    assert torch.equal(got[turns >= 32], base.float().double()[turns >= 32]) and keep.min() == 0
    for bad in (dict(rot=3), dict(rot=0), dict(rot=130), dict(rot=8, base=1.0), dict(rot=8, base=math.inf), dict(rot=8, factor=0.5),
                dict(rot=8, length=-1.0), dict(rot=8, length=64.0, slow_turns=3.0, fast_turns=3.0), dict(rot=8, base=math.nan),
                dict(rot=8, length=64.0, slow_turns=-1.0)):
        with pytest.raises(B.LLError):
            B.ll_rope_freqs(**bad)


def test_binding_refuses_tensors_that_are_not_on_the_gpu(B):
    q, v, g = torch.zeros(1, 2, 4, 16), torch.zeros(1, 2, 4, 16), torch.zeros(1, 2, 4)
    for f in (lambda: B.ll_la_fwd(q, q, v, g), lambda: B.ll_la_bwd(q, q, v, g, v),
              lambda: B.ll_la_decode_step(q[:, :, 0], q[:, :, 0], v[:, :, 0], g[:, :, 0], torch.zeros(1, 2, 16, 16)),
              lambda: B.ll_rope_fwd(q, None, torch.ones(4)), lambda: B.ll_rope_bwd(q, q, torch.ones(4))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError):
        B.make_la_shape(1, 1, 1, 1 << 32, 16, 16)
