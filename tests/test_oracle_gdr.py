"""The gated delta rule's oracle: against the dense form, against the
log-linear Gated DeltaNet with every lambda 1, and its gradient against
central differences.  And the host-side refusals of the ll_gdr_* entry points."""

import ctypes

import numpy as np
import pytest

from oracle import gdn, gdr
from oracle.partition import levels_needed


def _draw(T, dk, dv, seed, slow=False):
    r = np.random.default_rng(seed)
    k = r.standard_normal((T, dk))
    k /= np.linalg.norm(k, axis=1, keepdims=True)
    la = -np.log1p(np.exp(r.standard_normal(T) - (4 if slow else 0)))
    return r.standard_normal((T, dk)) / dk ** 0.5, k, r.standard_normal((T, dv)), la, 1 / (1 + np.exp(-r.standard_normal(T)))


@pytest.mark.parametrize("T", [1, 2, 7, 40])
def test_forward_is_the_dense_form(T):
    q, k, v, la, b = _draw(T, 8, 5, T)
    o, _ = gdr.forward(q, k, v, la, b, scale=0.5)
    assert np.allclose(o, 0.5 * gdn.gdn_coeff(q, k, b, la) @ v, atol=1e-12)
    ones = np.ones((T, levels_needed(T)))
    assert np.allclose(o, 0.5 * gdn.gdn_forward_A(q, k, v, b, la, ones), atol=1e-12)


def test_forward_continues_from_its_state():
    q, k, v, la, b = _draw(23, 8, 5, 3, slow=True)
    o, S = gdr.forward(q, k, v, la, b)
    o1, S1 = gdr.forward(q[:9], k[:9], v[:9], la[:9], b[:9])
    o2, S2 = gdr.forward(q[9:], k[9:], v[9:], la[9:], b[9:], state=S1)
    assert np.allclose(np.concatenate([o1, o2]), o, atol=1e-13) and np.allclose(S2, S, atol=1e-13)


def test_gradient_against_differences():
    T, dk, dv = 6, 4, 3
    q, k, v, la, b = _draw(T, dk, dv, 5, slow=True)
    r = np.random.default_rng(6)
    S0, do, dS = r.standard_normal((dv, dk)), r.standard_normal((T, dv)), r.standard_normal((dv, dk))
    x = dict(q=q, k=k, v=v, log_alpha=la, beta=b, state=S0)

    def f(**kw):
        o, S = gdr.forward(scale=0.7, **kw)
        return np.sum(o * do) + np.sum(S * dS)

    g = gdr.backward(q, k, v, la, b, do, scale=0.7, state=S0, dstate=dS)
    g["dstate"] = g.pop("dstate_in")
    h = 1e-5
    for n, a in x.items():
        for i in np.ndindex(a.shape):
            hi, lo = a.copy(), a.copy()
            hi[i] += h
            lo[i] -= h
            num = (f(**{**x, n: hi}) - f(**{**x, n: lo})) / (2 * h)
            # central differences: O(h^2) truncation and 1e-16 / h rounding of a value of order 10
            assert abs(num - g["d" + n][i]) <= 1e-7 * max(1.0, abs(num)), (n, i)


# ------------------------------------------------------------------ refusals, no GPU needed
FAKE = 0x7f0000000000  # never dereferenced: every call below fails a host-side check


@pytest.fixture(scope="module")
def B():
    import os

    from log_linear_attention_chunked_gb300 import binding
    if not os.path.exists(binding.LIB_PATH):
        from log_linear_attention_chunked_gb300 import build
        build.build()
    binding.lib()
    return binding


def _shape(lib_, **kw):
    d = dict(B=2, H=4, Hk=2, T=64, dk=16, dv=32, n_seqs=0, scale=1.0, io=lib_.LL_F32)
    d.update(kw)
    return lib_.make_gdr_shape(**d)


BAD_SHAPES = [(dict(B=0), 1), (dict(T=0), 1), (dict(H=0), 1), (dict(Hk=0), 1), (dict(Hk=3), 1), (dict(n_seqs=-1), 1),
              (dict(n_seqs=2), 1), (dict(io=5), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1),
              (dict(dk=96), 2), (dict(dv=8), 2), (dict(dv=256), 2), (dict(B=1 << 20, T=1 << 20), 2)]


def _ptrs(n):
    return [FAKE + (i << 36) for i in range(n)]


def _call(lib_, entry, shape, ptrs, ws=FAKE + (30 << 36), ws_bytes=1 << 50):
    vp = ctypes.c_void_p
    return getattr(lib_.lib(), entry)(ctypes.byref(shape), *[vp(x) if x else None for x in ptrs],
                                   vp(ws) if ws else None, ctypes.c_size_t(ws_bytes), None)


@pytest.mark.parametrize("kw,status", BAD_SHAPES)
def test_shapes_are_refused(B, kw, status):
    s = _shape(B, **kw)
    assert _call(B, "ll_gdr_fwd", s, [0] + _ptrs(8)) == status
    assert _call(B, "ll_gdr_bwd", s, [0] + _ptrs(14)) == status
    assert B.ll_gdr_bwd_workspace_size(s) == 0
    assert B.ll_gdr_fwd_launches(s) == 0 and B.ll_gdr_bwd_launches(s) == 0


def test_fwd_arguments_are_refused(B):
    s = _shape(B)
    # seq_starts, q, k, v, log_alpha, beta, state_in, o, state_out
    p = [0] + _ptrs(8)
    for i in (1, 2, 3, 4, 5, 7):
        assert _call(B, "ll_gdr_fwd", s, [0 if j == i else x for j, x in enumerate(p)]) == 1, i
    for i in range(1, 9):  # misaligned
        assert _call(B, "ll_gdr_fwd", s, [x + 8 if j == i else x for j, x in enumerate(p)]) == 1, i
    assert _call(B, "ll_gdr_fwd", s, [FAKE + (20 << 36)] + p[1:]) == 1          # starts without n_seqs
    assert _call(B, "ll_gdr_fwd", _shape(B, B=1, n_seqs=2), p) == 1             # n_seqs without starts
    assert _call(B, "ll_gdr_fwd", s, p[:7] + [p[3]] + p[8:]) == 1               # o on v
    assert _call(B, "ll_gdr_fwd", s, p[:8] + [p[6] + 16]) == 1                  # state_out inside state_in
    assert _call(B, "ll_gdr_fwd", s, p[:8] + [p[7]]) == 1                       # state_out on o


def test_fwd_workspace_is_refused(B):
    s = _shape(B, T=4096, dk=128, dv=128, io=B.LL_BF16)
    need = B.ll_gdr_fwd_workspace_size(s)
    if need:
        p = [0] + _ptrs(8)
        assert _call(B, "ll_gdr_fwd", s, p, ws=0) == 5
        assert _call(B, "ll_gdr_fwd", s, p, ws_bytes=need - 1) == 5
        assert _call(B, "ll_gdr_fwd", s, p, ws=FAKE + (30 << 36) + 128) == 5


def test_bwd_arguments_are_refused(B):
    s = _shape(B)
    # seq_starts, q, k, v, log_alpha, beta, state_in, dout, dstate_out, dq, dk, dv, dlog_alpha, dbeta, dstate_in
    p = [0] + _ptrs(14)
    for i in (1, 2, 3, 4, 5, 7, 9, 10, 11, 12, 13):
        assert _call(B, "ll_gdr_bwd", s, [0 if j == i else x for j, x in enumerate(p)]) == 1, i
    for i in range(1, 15):
        assert _call(B, "ll_gdr_bwd", s, [x + 4 if j == i else x for j, x in enumerate(p)]) == 1, i
    for i in (9, 10, 11, 12, 13, 14):  # an output on an input, and on the next output
        assert _call(B, "ll_gdr_bwd", s, [p[1] if j == i else x for j, x in enumerate(p)]) == 1, i
        assert _call(B, "ll_gdr_bwd", s, [p[9 + (i - 8) % 6] if j == i else x for j, x in enumerate(p)]) == 1, i
    assert _call(B, "ll_gdr_bwd", s, p, ws=0) == 5
    assert _call(B, "ll_gdr_bwd", s, p, ws_bytes=B.ll_gdr_bwd_workspace_size(s) - 1) == 5
    assert _call(B, "ll_gdr_bwd", s, p, ws=FAKE + (30 << 36) + 64) == 5


def test_decode_arguments_are_refused(B):
    vp, L = ctypes.c_void_p, B.lib()

    def step(Bn=2, H=4, Hk=2, dk=16, dv=16, io=0, scale=1.0, n=8, slots=FAKE + (20 << 36), p=None):
        p = p or _ptrs(7)  # q, k, v, log_alpha, beta, states, o
        return L.ll_gdr_decode_step(Bn, H, Hk, dk, dv, io, scale, vp(slots) if slots else None, n,
                                    *[vp(x) if x else None for x in p], None)

    assert step(Bn=0) == 1 and step(H=0) == 1 and step(Hk=0) == 1 and step(Hk=3) == 1 and step(n=0) == 1
    assert step(io=7) == 1 and step(scale=float("nan")) == 1
    assert step(dk=96) == 2 and step(dv=256) == 2 and step(Bn=1 << 20, H=1 << 10, n=1 << 20) == 2
    assert step(slots=0, n=1) == 1                       # fewer states than rows
    assert step(slots=FAKE + (20 << 36) + 8) == 1
    for i in range(7):
        p = _ptrs(7)
        assert step(p=[0 if j == i else x for j, x in enumerate(p)]) == 1, i
        assert step(p=[x + 8 if j == i else x for j, x in enumerate(p)]) == 1, i
    p = _ptrs(7)
    assert step(p=p[:6] + [p[2]]) == 1                   # o on v
    assert step(p=p[:5] + [p[1], p[6]]) == 1             # states on k
    assert step(p=p[:6] + [p[5] + 64]) == 1              # o inside the states


@pytest.mark.parametrize("T", [(1 << 31) - 1, (1 << 31) - 128])
def test_lengths_at_the_end_of_31_bits_are_refused(B, T):
    """One head: few enough CTAs, but a length rounded up to whole chunks passes 2^31."""
    for io in (B.LL_F32, B.LL_BF16):
        s = _shape(B, B=1, H=1, Hk=1, T=T, dk=16, dv=16, io=io)
        assert _call(B, "ll_gdr_fwd", s, [0] + [FAKE + (i << 40) for i in range(8)], ws=FAKE + (30 << 40)) == 2
        assert _call(B, "ll_gdr_bwd", s, [0] + [FAKE + (i << 40) for i in range(14)], ws=FAKE + (30 << 40)) == 2
        assert B.ll_gdr_bwd_workspace_size(s) == 0 and B.ll_gdr_fwd_launches(s) == 0


@pytest.mark.parametrize("name", ["B", "H", "Hk", "T", "dk", "dv", "n_seqs"])
def test_sizes_beyond_32_bits_are_refused(B, name):
    """Taken modulo 2^32 such a call would work on a few of its tokens and return."""
    with pytest.raises(ValueError):
        _shape(B, **{name: (1 << 32) + 16})
