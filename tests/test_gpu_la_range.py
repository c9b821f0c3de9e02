"""GPU parity of linear attention with a decay per head (ll_la_fwd, ll_la_bwd, ll_la_decode_step) against the
recurrence in 64 bits (oracle.la) where tests/test_gpu_la.py does not go: segments of many chunks, many heads, many
packed sequences, memory that changes within a segment, the accuracy of states and of the decays' gradients, starts out of order
over several launches, infinities, and far rotary positions.

Tolerances of outputs and states as there, but by the way that a call takes (chunks or token by token).

Tolerances of dlog_alpha.  A token's value is a sum of terms along the sequence, of products of v and dv (k and dk)
and of q and dq, from the nearer of the two ends of its piece: segments and tokens that forget.  With D the standard deviation of a
term's error relative to its size, the sum over n tokens is off by D sqrt(sum of squares) (2-norm), and over some ten
thousand tokens of a test no value by more than five times that; on top TOL_F32 of the largest term for the border's
own product, as in tests/test_gpu_la.py.  In chunks D is 5e-7 (test_decay_gradients_keep_float32), token by token it is
2^-22: a float32 product of 128 elements and the two sums that it is made of, each rounded by half of 2^-23, with a few of
the recurrence's own roundings."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import la
from tests._parity import TOL_BF16, TOL_F32, rel_err
from tests.test_gpu_la import B, DEV, check_bwd, check_fwd, draw, gpu_bwd, gpu_fwd, setup  # noqa: F401

pytestmark = pytest.mark.gpu
D_CHUNKS, D_TOKENS = 5e-7, 2.0 ** -22


def in_chunks(x, starts, bwd):
    """Does a call of these tensors go in chunks?  (bf16, 64 and 128, from some mean length on.)"""
    Bn, _, T, dk = x["q"].shape
    H, dv = x["v"].shape[1], x["v"].shape[3]
    if x["q"].dtype != torch.bfloat16 or min(dk, dv) < 64:
        return False
    n = Bn if starts is None else len(starts) - 1
    mean = T if starts is None else -(-T // n)
    few = n * H <= 152
    if dk != dv:
        return mean >= ((8 if bwd else 24) if few else 40)
    return mean >= ((48 if few else 24) if dk == 128 else (16 if few else 48) + (16 if bwd else 0))


def tol_out(x, starts, bwd):
    return TOL_F32 if x["q"].dtype == torch.float32 else TOL_BF16 if in_chunks(x, starts, bwd) else 2.0 ** -8 + TOL_F32


def head(x, starts, i, h):
    """What the oracle takes of sequence i and value head h, and where it stands."""
    b, lo, hi = (i, 0, x["q"].shape[2]) if starts is None else (0, starts[i], starts[i + 1])
    hk = h // (x["v"].shape[1] // x["q"].shape[1])
    f = {n: x[n][b, hk if n in "qk" else h, lo:hi].double().numpy() for n in ("q", "k", "v", "dout")}
    ga = x["log_alpha"]
    ga = np.full(hi - lo, float(ga[h])) if ga.dim() == 1 else ga[b, h, lo:hi].double().numpy()
    st, ds = [x[n][i, h].double().numpy() if n in x else None for n in ("state_in", "dstate_out")]
    return (b, hk, lo, hi), [f["q"], f["k"], f["v"], ga], f["dout"], st, ds


def squares(a, r):
    """The squares of a token's terms."""
    return (a[0] * r["dq"]).sum(-1) ** 2 + np.maximum((a[1] * r["dk"]).sum(-1) ** 2, (a[2] * r["dv"]).sum(-1) ** 2)


def check_heads(B, x, starts, which, scale=0.5):
    """Forward and gradient; the oracle on every value head of the key heads (sequence, key head) of `which`."""
    o, st = gpu_fwd(B, x, starts, scale)
    d = gpu_bwd(B, x, starts, scale)
    again = gpu_fwd(B, x, starts, scale), gpu_bwd(B, x, starts, scale)
    assert np.array_equal(o, again[0][0]) and np.array_equal(st, again[0][1])
    assert all(np.array_equal(p, q) for p, q in zip(d, again[1])), "two calls differ"
    dq, dk, dv, dla, dst = d
    G = x["v"].shape[1] // x["q"].shape[1]
    tf, tb = tol_out(x, starts, False), tol_out(x, starts, True)
    D = D_CHUNKS if in_chunks(x, starts, True) else D_TOKENS
    for i, key in which:
        rq = rk = 0.0
        for h in range(key * G, key * G + G):
            (b, hk, lo, hi), a, do, s0, ds = head(x, starts, i, h)
            ro, rs = la.forward(*a, scale=scale, state=s0)
            assert rel_err(st[i, h], rs, 0) <= TOL_F32, (i, h, "state")
            r = la.backward(*a, do, scale=scale, state=s0, dstate=ds)
            assert rel_err(dst[i, h], r["dstate_in"], 0) <= TOL_F32, (i, h, "dstate_in")
            if hi == lo:
                continue
            assert rel_err(o[b, h, lo:hi], ro, 0) <= tf, (i, h, "o")
            assert rel_err(dv[b, h, lo:hi], r["dv"], 0) <= tb, (i, h, "dv")
            rq, rk = rq + r["dq"], rk + r["dk"]
            if dla.ndim == 3:
                s2 = squares(a, r)
                bound = 5 * D * np.sqrt(s2.sum()) + TOL_F32 * max(np.sqrt(s2.max()), r["terms"].max())
                assert np.abs(dla[b, h, lo:hi] - r["dlog_alpha"]).max() <= bound, (i, h, "dlog_alpha")
        if hi > lo:
            assert rel_err(dq[b, hk, lo:hi], rq, 0) <= tb and rel_err(dk[b, hk, lo:hi], rk, 0) <= tb, (i, key, "dq, dk")


# ---------------------------------------------------------------- segments of many chunks, many heads, many sequences
def most_segments(B, x, starts, bwd):
    """No more segments than this, in all sequences: by the states that the workspace holds."""
    _, (n, H, dv, dk), shape, _ = setup(B, {m: t for m, t in x.items() if m in ("q", "k", "v", "log_alpha")}, starts, 0.5)
    Bn, Hk, T = x["q"].shape[0], x["q"].shape[1], x["q"].shape[2]
    if not bwd:
        return B.ll_la_fwd_workspace_size(shape) // (H * dv * dk * 4)
    rest = Bn * H * T * 4 * (4 + (2 * dk if H != Hk else 0)) + n * H * dv * dk * 4
    return (B.ll_la_bwd_workspace_size(shape) - rest) // (2 * H * dv * dk * 4)


LONG = [  # B, H, Hk, T, dk, dv, starts, chunks of a segment (forward, gradient; at least), (sequence, key head) looked at
    (2, 16, 16, 4096, 128, 128, None, 4, 6, [(0, 0), (1, 15)]),
    (2, 16, 8, 4096, 128, 128, None, 4, 6, [(1, 3)]),
    (2, 32, 32, 3071, 64, 64, None, 4, 6, [(0, 1), (1, 31)]),
    (2, 16, 16, 3500, 64, 128, None, 4, 4, [(1, 2)]),
    (1, 16, 8, 7001, 128, 128, [3, 2600, 2601, 2601, 6200, 6999], 3, 4, [(0, 0), (3, 7), (4, 5)]),
    (1, 16, 16, 9000, 128, 64, [0, 4500, 9000], 4, 4, [(1, 9)]),
]


@pytest.mark.parametrize("case", LONG, ids=str)
def test_segments_of_many_chunks(B, case):  # noqa: F811
    """Slow decays: what a segment's later chunks hold and hand on is made of all of its chunks."""
    Bn, H, Hk, T, dk, dv, starts, fwd, bwd, which = case
    x = draw(Bn, H, Hk, T, dk, dv, "bf16", n=Bn if starts is None else len(starts) - 1, seed=T, rate=1e-3)
    chunks = Bn * -(-T // 128)
    assert chunks // most_segments(B, x, starts, False) >= fwd, "the case no longer has long segments"
    assert chunks // most_segments(B, x, starts, True) >= bwd, "the case no longer has long segments"
    check_heads(B, x, starts, which)


@pytest.mark.parametrize("T", [7, 8, 15, 16, 23, 24, 31, 39, 40, 47, 48, 63, 64])
@pytest.mark.parametrize("kind", [(154, 64, 64), (154, 128, 128), (76, 64, 128), (154, 128, 64), (2, 64, 128), (2, 64, 64), (2, 128, 128)], ids=str)
def test_short_sequences_of_many_heads(B, kind, T):  # noqa: F811
    """Both sides of the lengths from which chunks are taken, gradients too."""
    H, dk, dv = kind
    x = draw(2 if H == 76 else 1, H, H // 2, T, dk, dv, "bf16", seed=100 + T)
    check_heads(B, x, None, [(0, 0), (0, H // 2 - 1)])


@pytest.mark.parametrize("kind", [(4, 2, 128, 128, "bf16"), (2, 2, 128, 128, "f32"), (4, 4, 64, 64, "bf16")], ids=str)
def test_many_packed_sequences_token_by_token(B, kind):  # noqa: F811
    """Sequences of 0 to 15 tokens, more of them than a segment holds."""
    H, Hk, dk, dv, io = kind
    lens = [(7 * i) % 16 for i in range(260)]
    starts = np.concatenate([[0], np.cumsum(lens)]).tolist()
    T = starts[-1] + 3
    for per_head in (False, True):
        x = draw(1, H, Hk, T, dk, dv, io, n=len(lens), seed=71, per_head=per_head)
        assert not in_chunks(x, starts, True) and B.ll_la_fwd_launches(setup(B, x, starts, 0.5)[2]) == 3
        check_heads(B, x, starts, [(i, i % Hk) for i in (0, 1, 7, 16, 30, 128, 255, 258, 259)])
    check_fwd(B, x, starts)
    check_bwd(B, x, starts)


# ---------------------------------------------------------------- memory that changes within a segment
@pytest.mark.parametrize("kind", [(2, 16, 16, 128, 128, "bf16"), (2, 16, 8, 64, 64, "bf16"), (4, 16, 16, 128, 128, "f32"),
                                  (1, 2, 1, 32, 16, "f32"), (1, 2, 2, 64, 128, "bf16"), (8, 80, 80, 16, 16, "f32")], ids=str)
@pytest.mark.parametrize("how", ["forgets", "shortens", "forgets and grows"])
def test_decay_gradients_after_large_values(B, how, kind):  # noqa: F811
    """A long memory of values 256 times as large comes before (behind) a short one.  The gradients of the short one's
    decays are held to its own terms."""
    Bn, H, Hk, dk, dv, io = kind
    T, at = 3000, 1700
    x = draw(Bn, H, Hk, T, dk, dv, io, seed=81, init=how == "shortens", rate=1e-3)
    big, small = (slice(at, T), slice(0, at)) if how == "forgets and grows" else (slice(0, at), slice(at, T))
    x["v"][:, :, big] *= 256
    x["log_alpha"][:, :, small] = -torch.empty(Bn, H, T)[:, :, small].uniform_(0.7, 1.3, generator=torch.Generator().manual_seed(3))
    if how != "shortens":
        x["log_alpha"][:, :, at] = -float("inf")
    dla = gpu_bwd(B, x)[3]
    D = D_CHUNKS if in_chunks(x, None, True) else D_TOKENS
    for b, h in ((0, 0), (Bn - 1, H - 1)):
        _, a, do, s0, ds = head(x, None, b, h)
        r = la.backward(*a, do, scale=0.5, state=s0, dstate=ds)
        # (30 tokens at e^-1 leave e^-30 of the large values)
        part = slice(at + 30, T) if how == "shortens" else small
        s2 = squares(a, r)[part]
        bound = 5 * D * np.sqrt(s2.sum()) + TOL_F32 * max(np.sqrt(s2.max()), r["terms"][part].max())
        err = np.abs(dla[b, h] - r["dlog_alpha"])
        assert err[part].max() <= bound, (b, h, err[part].max() / bound)
        s2 = squares(a, r)
        assert err.max() <= 5 * D * np.sqrt(s2.sum()) + TOL_F32 * max(np.sqrt(s2.max()), r["terms"].max())


@pytest.mark.parametrize("kind", [(2, 16, 16, 128, 128, "bf16"), (1, 2, 1, 64, 64, "bf16"), (4, 16, 16, 128, 128, "f32"),
                                  (1, 3, 3, 16, 32, "f32"), (8, 80, 40, 16, 16, "bf16")], ids=str)
def test_tokens_that_forget_keep_pieces_apart(B, kind):  # noqa: F811
    """Pieces between tokens that forget, some of one token, with values from 2^-12 to 2^12: each held to its own terms."""
    Bn, H, Hk, dk, dv, io = kind
    T = 2500
    x = draw(Bn, H, Hk, T, dk, dv, io, seed=82, rate=0.02)
    cuts = [1, 2, 3, 40, 127, 128, 129, 300, 301, 600, 640, 1023, 1024, 1400, 1402, 1900, 2300, 2499]
    for n, (lo, hi) in enumerate(zip([0] + cuts, cuts + [T])):
        x["v"][:, :, lo:hi] *= 2.0 ** ((n * 7) % 25 - 12)
    x["state_in"] *= 1000
    x["dstate_out"] *= 1000
    x["log_alpha"][:, :, cuts] = -float("inf")
    dla = gpu_bwd(B, x)[3]
    D = D_CHUNKS if in_chunks(x, None, True) else D_TOKENS
    for b, h in ((0, 0), (Bn - 1, H - 1)):
        _, a, do, s0, ds = head(x, None, b, h)
        r = la.backward(*a, do, scale=0.5, state=s0, dstate=ds)
        s2 = squares(a, r)
        assert (dla[b, h, cuts] == 0).all()
        for lo, hi in zip([0] + cuts, cuts + [T]):
            bound = 5 * D * np.sqrt(s2[lo:hi].sum()) + TOL_F32 * max(np.sqrt(s2[lo:hi].max()), r["terms"][lo:hi].max())
            assert np.abs(dla[b, h, lo:hi] - r["dlog_alpha"][lo:hi]).max() <= bound, (b, h, lo)


@pytest.mark.parametrize("kind", [(1, 2, 2, 77, 128, 128, None), (1, 2, 1, 1000, 128, 64, None), (1, 2, 2, 2100, 64, 64, None),
                                  (2, 2, 1, 500, 64, 128, None), (1, 2, 1, 1300, 128, 128, [0, 5, 700, 700, 1297])], ids=str)
def test_states_keep_float32(B, kind):  # noqa: F811
    """What leaves a call as float32 is a sum of float32: products of three bf16 parts are exact to 2^-24, the tensor
    cores' eight steps of a chunk are cut off by 2^-24 of the sum so far on average (3.3e-7 as that grows like the root of
    the steps), and weights and additions round by 2^-24.  Twice that, 2-norm, is allowed: 1e-6.  (Two parts: 2.4e-6.)"""
    Bn, H, Hk, T, dk, dv, starts = kind
    x = draw(Bn, H, Hk, T, dk, dv, "bf16", n=Bn if starts is None else len(starts) - 1, seed=86, rate=0.01)
    assert in_chunks(x, starts, True)
    st, dst = gpu_fwd(B, x, starts)[1], gpu_bwd(B, x, starts)[4]
    for i in range(len(st)):
        for h in range(H):
            _, a, do, s0, ds = head(x, starts, i, h)
            want = la.forward(*a, scale=0.5, state=s0)[1]
            assert np.linalg.norm(st[i, h] - want) <= 1e-6 * np.linalg.norm(want), (i, h, "state_out")
            want = la.backward(*a, do, scale=0.5, state=s0, dstate=ds)["dstate_in"]
            assert np.linalg.norm(dst[i, h] - want) <= 1e-6 * np.linalg.norm(want), (i, h, "dstate_in")


@pytest.mark.parametrize("kind", [(2, 4, 4, 105, 128, 128, None, False, True), (1, 4, 2, 340, 128, 128, [0, 100, 220, 340], True, False),
                                  (3, 8, 4, 128, 64, 128, None, True, True), (2, 4, 4, 121, 64, 64, None, False, True),
                                  (1, 2, 2, 90, 128, 64, None, True, False)], ids=str)
def test_decay_gradients_keep_float32(B, kind):  # noqa: F811
    """Sequences of one chunk, whose two ends are known.  A term is a product of float32 values, the tensor cores' sum cut
    off as in test_states_keep_float32, and rounded a few times by 2^-24: 5e-7.  With independent errors, L of them squared on a
    token's left and R on its right, the joined sum is off by the root of L R / (L + R); a border's product of a state and
    a gradient, each within 1.7e-7, by 2.5e-7 of its terms, which every token shares.  All 2-norms over the tokens.
    (Terms from states in two bf16 parts, 1.6e-6, do not pass.)"""
    Bn, H, Hk, T, dk, dv, starts, init, final = kind
    x = draw(Bn, H, Hk, T, dk, dv, "bf16", n=Bn if starts is None else len(starts) - 1, seed=87, rate=0.05)
    assert in_chunks(x, starts, True)
    for n, there in (("state_in", init), ("dstate_out", final)):
        if not there:
            del x[n]
    dla = gpu_bwd(B, x, starts)[3]
    for i in range(Bn if starts is None else len(starts) - 1):
        for h in range(H):
            (b, _, lo, hi), a, do, s0, ds = head(x, starts, i, h)
            r = la.backward(*a, do, scale=0.5, state=s0, dstate=ds)
            left = np.concatenate([[0.0], np.cumsum(squares(a, r))])[:-1]
            right = squares(a, r).sum() - left
            ends = max(r["terms"][0], np.linalg.norm(la.forward(*a, scale=0.5, state=s0)[1] * (0.0 if ds is None else ds)))
            err = np.linalg.norm(dla[b, h, lo:hi] - r["dlog_alpha"])
            bound = 5e-7 * np.sqrt((left * right / (left + right)).sum()) + 2.5e-7 * ends * np.sqrt(hi - lo)
            assert err <= bound, (i, h)


@pytest.mark.parametrize("rate", [0.02, 2.0])
@pytest.mark.parametrize("kind", [(4, 2, 300, 128, 128, "bf16"), (4, 4, 256, 64, 64, "bf16"), (4, 2, 200, 32, 32, "f32")], ids=str)
def test_gradients_of_constant_decays(B, kind, rate):  # noqa: F811
    """The sum of a head's tokens.  A term's error goes to every token behind it, less the part that the joining of
    both sums takes back: to as many tokens as lie behind, minus the sum over all of them of the share of squares on their left."""
    H, Hk, T, dk, dv, io = kind
    x = draw(1, *kind, seed=88, per_head=True, rate=rate)
    seg, D = (128, D_CHUNKS) if in_chunks(x, None, True) else (64, D_TOKENS)
    dla = gpu_bwd(B, x)[3]
    for h in range(H):
        _, a, do, s0, ds = head(x, None, 0, h)
        r = la.backward(*a, do, scale=0.5, state=s0, dstate=ds)
        s2, var = squares(a, r), 0.0
        for lo in range(0, T, seg):
            w = s2[lo:lo + seg]
            before = np.concatenate([[0.0], np.cumsum(w)])[:-1]
            share = (before / w.sum()).sum()
            var += (w * (len(w) - 1 - np.arange(len(w)) - share) ** 2).sum()
        ends = max(r["terms"].max(), np.linalg.norm(la.forward(*a, scale=0.5, state=s0)[1] * ds))
        bound = 5 * D * np.sqrt(var) + 2.5e-7 * ends * T + 2.0 ** -23 * abs(r["dlog_alpha"].sum())
        assert abs(dla[h] - r["dlog_alpha"].sum()) <= bound, h


@pytest.mark.parametrize("kind", [(1, 2, 1, 100, 128, 128, "bf16", None), (3, 2, 2, 40, 32, 32, "f32", None), (2, 4, 2, 7, 64, 64, "bf16", None),
                                  (1, 2, 1, 100, 64, 128, "bf16", [0, 0, 40, 97, 97]), (1, 2, 1, 60, 16, 32, "f32", [5, 30, 30, 60]),
                                  (1, 2, 1, 900, 128, 128, "bf16", [0, 0, 400, 900])], ids=str)
def test_state_gradients_in_place(B, kind):  # noqa: F811
    """dstate_in in dstate_out's place, of one segment (the gradient there is read once more, for the decays') and of several."""
    Bn, H, Hk, T, dk, dv, io, starts = kind
    x = draw(Bn, H, Hk, T, dk, dv, io, n=Bn if starts is None else len(starts) - 1, seed=89)
    g, st_shape, _, ss = setup(B, x, starts, 0.5)
    a = (g["q"], g["k"], g["v"], g["log_alpha"], g["dout"])
    for state in (g["state_in"], None):
        apart, place = torch.empty(st_shape, device=DEV), g["dstate_out"].clone()
        grads = [torch.zeros_like(t) for t in a[:4]], [torch.zeros_like(t) for t in a[:4]]
        B.ll_la_bwd(*a, state_in=state, dstate_out=g["dstate_out"], dstate_in=apart, seq_starts=ss, grads=grads[0])
        B.ll_la_bwd(*a, state_in=state, dstate_out=place, dstate_in=place, seq_starts=ss, grads=grads[1])
        assert torch.equal(apart, place) and all(torch.equal(p, q) for p, q in zip(*grads))
        if starts is not None:
            for i in range(len(starts) - 1):
                assert starts[i] < starts[i + 1] or torch.equal(place[i], g["dstate_out"][i])
    check_bwd(B, x, starts)


# ---------------------------------------------------------------- bad starts
def test_starts_out_of_order_in_chunks(B):  # noqa: F811
    """Every launch of a call in chunks, over several segments: the error word, nothing outside of the buffers, and the next
    call is right."""
    T, H, Hk, d = 5000, 4, 2, 128
    x = draw(1, H, Hk, T, d, d, "bf16", n=3, seed=91)
    g, st_shape, shape, _ = setup(B, x, [0, 100, 200, T], 0.5)
    assert B.ll_la_fwd_launches(shape) == 3 and in_chunks(x, [0, 100, 200, T], True)
    for starts in ([0, 4000, 1000, T], [0, 1000, T + 1, T], [-5, 1000, 2000, T], [T, 3000, 2000, 0], [0, T, 0, T]):
        ss = torch.tensor(starts, dtype=torch.int32, device=DEV)
        for per_head in (False, True):
            ga = g["log_alpha"][0, :, 0].contiguous() if per_head else g["log_alpha"]
            st = torch.empty(st_shape, device=DEV)
            B.ll_la_fwd(g["q"], g["k"], g["v"], ga, state_in=g["state_in"], state_out=st, seq_starts=ss)
            assert B.ll_last_device_error() == 6, starts
            B.ll_la_bwd(g["q"], g["k"], g["v"], ga, g["dout"], state_in=g["state_in"], dstate_out=g["dstate_out"], dstate_in=st, seq_starts=ss)
            assert B.ll_last_device_error() == 6, starts
    check_heads(B, x, [0, 1700, 1700, 4990], [(0, 0), (1, 1), (2, 1)])


# ---------------------------------------------------------------- infinities
def test_infinite_states_stay_infinite(B):  # noqa: F811
    """Token by token a decay above zero times infinity is infinity, near one as elsewhere."""
    d = 32
    for rate in (0.0, 1e-6, 0.1, 0.49, 0.51, 3.0):
        g = {n: t.to(DEV) for n, t in draw(1, 2, 1, 1, d, d, "f32", seed=92, rate=rate, per_head=True).items()}
        st = torch.randn(1, 2, d, d, device=DEV)
        st[0, 0, 3, 4], st[0, 1, 5, 6] = float("inf"), -float("inf")
        a = [g[n][:, :, 0].contiguous() for n in ("q", "k", "v")]
        pool = st.clone()
        B.ll_la_decode_step(*a, g["log_alpha"], pool)
        out = torch.empty_like(st)
        B.ll_la_fwd(g["q"], g["k"], g["v"], g["log_alpha"], state_in=st, state_out=out)
        for x in (pool, out):
            assert x[0, 0, 3, 4] == float("inf") and x[0, 1, 5, 6] == -float("inf"), rate
            assert torch.isfinite(x).sum() == x.numel() - 2
    # over segments: the state on entry to the second
    T = 300
    g = {n: t.to(DEV) for n, t in draw(1, 1, 1, T, d, d, "f32", seed=93, rate=1e-3, per_head=True).items()}
    g["state_in"][0, 0, 3, 4] = float("inf")
    g["dstate_out"][0, 0, 5, 6] = -float("inf")
    out, back = torch.empty_like(g["state_in"]), torch.empty_like(g["state_in"])
    B.ll_la_fwd(g["q"], g["k"], g["v"], g["log_alpha"], state_in=g["state_in"], state_out=out)
    B.ll_la_bwd(g["q"], g["k"], g["v"], g["log_alpha"], g["dout"], dstate_out=g["dstate_out"], dstate_in=back)
    assert out[0, 0, 3, 4] == float("inf") and back[0, 0, 5, 6] == -float("inf")


# ---------------------------------------------------------------- far rotary positions
PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


def test_rope_angles_at_the_farthest_positions(B):  # noqa: F811
    """The angle is off by 2^-32 of a turn from its last bits and by |position| 2^-65 from the frequency's rounding to 2^-64
    of a turn; sine and cosine by 3 x 2^-24 on top."""
    f = torch.cat([B.ll_rope_freqs(56), torch.tensor([1.9, 2.5, 0.77, 6.2831855])])
    places = [1 << 32, (1 << 33) - 7, 1 << 36, -(1 << 40) + 3, 1 << 40, 1 << 44, 5 << 41]
    x = torch.zeros(1, 1, len(places), 64)
    x[..., :32] = 1.0
    got = B.ll_rope_fwd(x.to(DEV), None, f.to(DEV), positions=torch.tensor([places], device=DEV)).double().cpu().numpy()[0, 0]
    for n, pos in enumerate(places):
        turns = [Fraction(float(w)) * pos / (2 * PI) for w in f]
        angle = np.array([float((t - round(t)) * 2 * PI) for t in turns])
        err = max(np.abs(got[n, :32] - np.cos(angle)).max(), np.abs(got[n, 32:] - np.sin(angle)).max())
        assert err <= 2 * np.pi * (2.0 ** -32 + 1.001 * abs(pos) * 2.0 ** -65) + 3 * 2.0 ** -24, (pos, err)
