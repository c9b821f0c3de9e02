"""GPU parity of linear attention with a decay per head (ll_la_fwd, ll_la_bwd,
ll_la_decode_step) and of rotary positions (ll_rope_fwd, ll_rope_bwd) against the
recurrence in 64 bits (oracle.la).

Tolerances, relative to a (sequence, head) slice's largest value.  float32
values: TOL_F32, as every float32 path here (rounding of float32 sums).  bf16
outputs of float32 arithmetic (the token-by-token path, the decode step, the
rotations): half a step of bf16, 2^-8, on top of that.  bf16 outputs of the tensor-core
path, whose operands (states, masked scores) are rounded to 16 bits once each: TOL_BF16,
as every bf16 tensor-core path here.  Decays' gradients are sums that may cancel: TOL_F32
relative to their terms.  These are the products of q and dq, k and dk, and those of the definition,
sum_ab (alpha S_{t-1})_ab (A_t)_ab: with both factors off by independent relative errors d the sum is off
by sqrt(2) d |S * A| (2-norm), and states of the tensor-core path, whose operands have two bf16 parts, by
d <= 2^-18 from each rounding (rms 1.6e-6): sqrt(2) 1.6e-6 |S * A| is a quarter of TOL_F32 |S * A|."""

import numpy as np
import pytest
import torch

from oracle import la
from tests._parity import TOL_BF16, TOL_F32, Guarded, rel_err

pytestmark = pytest.mark.gpu
DEV = "cuda"
SEVEN = torch.tensor(7.0)


@pytest.fixture(scope="module")
def B():
    from log_linear_attention_chunked_gb300 import binding
    binding.lib()
    return binding


def draw(Bn, H, Hk, T, dk, dv, io="bf16", n=None, seed=0, init=True, per_head=False, rate=None):
    """CPU tensors of one call; n: states (sequences)."""
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32

    def r(*s):
        return torch.randn(*s, generator=g)

    rate = torch.logspace(-2.7, 0.3, H) if rate is None else torch.full((H,), rate)
    x = dict(q=r(Bn, Hk, T, dk).to(dt), k=r(Bn, Hk, T, dk).to(dt), v=r(Bn, H, T, dv).to(dt),
             log_alpha=-rate if per_head else -rate.view(1, H, 1) * torch.nn.functional.softplus(r(Bn, H, T)),
             dout=r(Bn, H, T, dv).to(dt))
    if init:
        x["state_in"] = r(n or Bn, H, dv, dk)
        x["dstate_out"] = r(n or Bn, H, dv, dk)
    return x


def seqs_of(x, starts):
    """(state row, batch row, first, end) of every sequence."""
    Bn, _, T, _ = x["q"].shape
    return [(b, b, 0, T) for b in range(Bn)] if starts is None else [(i, 0, starts[i], starts[i + 1])
                                                                    for i in range(len(starts) - 1)]


def slices(x, starts):
    H, Hk = x["v"].shape[1], x["q"].shape[1]
    f = {n: t.double().numpy() for n, t in x.items()}
    for i, b, lo, hi in seqs_of(x, starts):
        for h in range(H):
            hk = h // (H // Hk)
            ga = np.full(hi - lo, f["log_alpha"][h]) if f["log_alpha"].ndim == 1 else f["log_alpha"][b, h, lo:hi]
            a = [f["q"][b, hk, lo:hi], f["k"][b, hk, lo:hi], f["v"][b, h, lo:hi], ga]
            st = f["state_in"][i, h] if "state_in" in f else None
            ds = f["dstate_out"][i, h] if "dstate_out" in f else None
            yield (i, b, h, hk, lo, hi), a, f["dout"][b, h, lo:hi], st, ds


def setup(B, x, starts, scale):
    g = {n: t.to(DEV) for n, t in x.items()}
    Bn, Hk, T, dk = g["q"].shape
    _, H, _, dv = g["v"].shape
    n = Bn if starts is None else len(starts) - 1
    shape = B.make_la_shape(Bn, H, Hk, T, dk, dv, 0 if starts is None else n, scale, B._io(g["q"].dtype), x["log_alpha"].dim() == 1)
    return g, (n, H, dv, dk), shape, None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)


def gpu_fwd(B, x, starts=None, scale=0.5):
    g, st_shape, shape, ss = setup(B, x, starts, scale)
    o, st = Guarded(tuple(g["v"].shape), g["v"].dtype, fill=SEVEN), Guarded(st_shape, torch.float32)
    ws = Guarded((max(256, B.ll_la_fwd_workspace_size(shape)),), torch.uint8)
    B.ll_la_fwd(g["q"], g["k"], g["v"], g["log_alpha"], scale=scale, state_in=g.get("state_in"), state_out=st.view,
                seq_starts=ss, o=o.view, workspace=ws.view)
    assert B.ll_last_device_error() == 0
    assert o.intact() and st.intact() and ws.intact(), "write outside a buffer"
    return o.view.float().cpu().numpy(), st.view.cpu().numpy()


def tensor_cores(x):
    return x["q"].dtype == torch.bfloat16 and x["q"].shape[3] >= 64 and x["v"].shape[3] >= 64


def tol_out(x):
    return TOL_F32 if x["q"].dtype == torch.float32 else TOL_BF16 if tensor_cores(x) else 2.0 ** -8 + TOL_F32


def check_fwd(B, x, starts=None, scale=0.5):
    o, st = gpu_fwd(B, x, starts, scale)
    covered = np.zeros(o.shape, bool)
    for (i, b, h, hk, lo, hi), a, _, s0, _ in slices(x, starts):
        ro, rs = la.forward(*a, scale=scale, state=s0)
        covered[b, h, lo:hi] = True
        assert rel_err(st[i, h], rs, 0) <= TOL_F32, (i, h, "state")
        if hi > lo:
            assert rel_err(o[b, h, lo:hi], ro, 0) <= tol_out(x), (i, h, "o")
    assert (o[~covered] == 7.0).all(), "a row outside every sequence was written"


def gpu_bwd(B, x, starts=None, scale=0.5):
    g, st_shape, shape, ss = setup(B, x, starts, scale)
    out = [Guarded(tuple(g[s].shape), g[s].dtype, fill=SEVEN) for s in ("q", "k", "v", "log_alpha")]
    ds = Guarded(st_shape, torch.float32)
    ws = Guarded((B.ll_la_bwd_workspace_size(shape),), torch.uint8)
    B.ll_la_bwd(g["q"], g["k"], g["v"], g["log_alpha"], g["dout"], scale=scale, state_in=g.get("state_in"),
                dstate_out=g.get("dstate_out"), seq_starts=ss, grads=[t.view for t in out], dstate_in=ds.view, workspace=ws.view)
    assert B.ll_last_device_error() == 0
    assert all(t.intact() for t in out) and ds.intact() and ws.intact(), "write outside a buffer"
    return [t.view.float().cpu().numpy() for t in out] + [ds.view.cpu().numpy()]


def check_bwd(B, x, starts=None, scale=0.5):
    dq, dk, dv, dla, dst = gpu_bwd(B, x, starts, scale)
    rq, rk = np.full(dq.shape, 7.0), np.full(dk.shape, 7.0)
    covered = np.zeros(dv.shape[:3], bool)
    for i, b, lo, hi in seqs_of(x, starts):
        rq[b, :, lo:hi] = rk[b, :, lo:hi] = 0.0
    whole, terms = np.zeros(dv.shape[1]), np.zeros(dv.shape[1])
    for (i, b, h, hk, lo, hi), a, do, s0, ds in slices(x, starts):
        r = la.backward(*a, do, scale=scale, state=s0, dstate=ds)
        assert rel_err(dst[i, h], r["dstate_in"], 0) <= TOL_F32, (i, h, "dstate_in")
        covered[b, h, lo:hi] = True
        if hi == lo:
            continue
        rq[b, hk, lo:hi] += r["dq"]
        rk[b, hk, lo:hi] += r["dk"]
        assert rel_err(dv[b, h, lo:hi], r["dv"], 0) <= tol_out(x), (i, h, "dv")
        term = max(np.abs((a[0] * r["dq"]).sum(-1)).max(), np.abs((a[1] * r["dk"]).sum(-1)).max(), r["terms"].max())
        if dla.ndim == 1:
            whole[h] += r["dlog_alpha"].sum()
            # a token's value may be off by TOL_F32 term; those of neighbours share their sums (dlog_alpha_t and
            # dlog_alpha_{t+1} differ by one token's terms), so their errors are equal rather than
            # independent and the bound of the sum over a sequence is that of its tokens, added up
            terms[h] += term * (hi - lo)
        else:
            assert np.abs(dla[b, h, lo:hi] - r["dlog_alpha"]).max() <= TOL_F32 * max(term, 1e-30), (i, h, "dlog_alpha")
    if dla.ndim == 1:
        assert (np.abs(dla - whole) <= TOL_F32 * np.maximum(np.maximum(terms, np.abs(whole)), 1e-30)).all(), "dlog_alpha"
    for name, got, ref in (("dq", dq, rq), ("dk", dk, rk)):
        for i, b, lo, hi in seqs_of(x, starts):
            if hi > lo:
                assert rel_err(got[b, :, lo:hi], ref[b, :, lo:hi], 1) <= tol_out(x), (i, name)
    assert (dv[~covered] == 7.0).all()
    assert dla.ndim == 1 or (dla[~covered] == 7.0).all()
    Hk, H = dq.shape[1], dv.shape[1]
    un = ~covered[:, ::H // Hk]
    assert (dq[un] == 7.0).all() and (dk[un] == 7.0).all(), "a row outside every sequence was written"


SHAPES = [  # B, H, Hk, T, dk, dv, io
    (1, 1, 1, 1, 16, 16, "f32"), (2, 2, 1, 2, 32, 16, "f32"), (1, 2, 2, 15, 16, 32, "bf16"), (1, 4, 2, 17, 16, 128, "f32"),
    (2, 4, 1, 33, 128, 16, "f32"), (1, 2, 1, 65, 64, 64, "f32"), (1, 2, 2, 130, 128, 128, "f32"), (3, 2, 2, 257, 32, 64, "bf16"),
    (1, 1, 1, 700, 16, 16, "bf16"), (1, 2, 1, 333, 64, 32, "f32"),
    # tensor cores
    (1, 2, 1, 1, 128, 128, "bf16"), (2, 2, 2, 16, 64, 64, "bf16"), (1, 2, 1, 127, 128, 64, "bf16"), (1, 2, 2, 128, 64, 128, "bf16"),
    (2, 2, 1, 129, 128, 128, "bf16"), (1, 4, 2, 300, 128, 128, "bf16"), (1, 2, 1, 640, 64, 64, "bf16"), (1, 3, 3, 1100, 128, 128, "bf16"),
    (1, 1, 1, 2200, 64, 128, "bf16"),
]


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(B, shape, per_head):
    check_fwd(B, draw(*shape, seed=1, per_head=per_head))


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(B, shape, per_head):
    check_bwd(B, draw(*shape, seed=2, per_head=per_head))


PACKED = [  # starts, T: empty sequences, single tokens, rows before, between and behind the sequences
    ([0, 5, 5, 6, 70], 70), ([3, 3, 40, 168, 296, 297, 560], 600), ([0, 1], 1), ([0, 0, 0], 4), ([7, 135, 300, 300], 301),
    (list(range(0, 41)), 41), ([0, 1300, 1301, 1301, 1500], 1503),
    ([0, 1, 2, 3, 5, 5, 8, 700, 829], 829), ([2, 130, 258, 259, 515, 515, 643], 700),
]


@pytest.mark.parametrize("kind", [(2, 1, 128, 128, "bf16"), (2, 2, 64, 64, "bf16"), (4, 2, 32, 64, "f32"), (2, 1, 64, 128, "bf16")], ids=str)
@pytest.mark.parametrize("starts,T", PACKED, ids=[str(i) for i in range(len(PACKED))])
def test_packed(B, starts, T, kind):
    H, Hk, dk, dv, io = kind
    for per_head in (False, True):
        x = draw(1, H, Hk, T, dk, dv, io, n=len(starts) - 1, seed=T, per_head=per_head)
        check_fwd(B, x, starts)
        check_bwd(B, x, starts)


@pytest.mark.parametrize("kind", [(2, 1, 300, 128, 128, "bf16"), (2, 2, 150, 32, 32, "f32"), (2, 1, 140, 64, 64, "bf16")], ids=str)
def test_without_states(B, kind):
    x = draw(1, *kind, seed=5, init=False)
    check_fwd(B, x)
    check_bwd(B, x)
    y = dict(x, dstate_out=torch.randn(1, kind[0], kind[4], kind[3], generator=torch.Generator().manual_seed(1)))
    check_bwd(B, y)
    y = dict(x, state_in=y["dstate_out"])
    check_bwd(B, y)


@pytest.mark.parametrize("kind", [(2, 1, 128, 128, "bf16"), (2, 2, 32, 32, "f32"), (2, 2, 64, 64, "bf16")], ids=str)
@pytest.mark.parametrize("rate", [0.0, 1e-7, 4.0, 30.0, 200.0])
def test_decays_from_none_to_all(B, rate, kind):
    H, Hk, dk, dv, io = kind
    for per_head in (False, True):
        x = draw(1, H, Hk, 400, dk, dv, io, seed=7, per_head=per_head, rate=rate)
        check_fwd(B, x)
        check_bwd(B, x)


@pytest.mark.parametrize("kind", [(2, 1, 128, 128, "bf16"), (2, 2, 32, 32, "f32"), (2, 1, 64, 64, "bf16")], ids=str)
def test_tokens_that_forget(B, kind):
    """log alpha = -inf: the state is forgotten, and its logarithm has no gradient."""
    H, Hk, dk, dv, io = kind
    x = draw(1, H, Hk, 500, dk, dv, io, seed=8)
    for t in (0, 1, 63, 127, 128, 129, 200, 201, 202, 383, 499):
        x["log_alpha"][:, :, t] = -float("inf")
    check_fwd(B, x)
    check_bwd(B, x)
    x["log_alpha"][:] = -float("inf")
    check_fwd(B, x)
    check_bwd(B, x)


@pytest.mark.parametrize("kind", [(1, 1, 128, 128, "bf16"), (1, 1, 32, 16, "f32")], ids=str)
def test_constant_decays_do_not_drift(B, kind):
    """A decay of e^-1 over the sequence, in 20000 equal steps, and a state that it carries."""
    H, Hk, dk, dv, io = kind
    T = 20000
    x = draw(1, H, Hk, T, dk, dv, io, seed=9, per_head=True, rate=1.0 / T)
    for n in ("q", "k", "v"):
        x[n][:, :, :-1] = 0
    o, st = gpu_fwd(B, x)
    s0 = x["state_in"][0, 0].double().numpy()
    want = np.exp(T * x["log_alpha"].double().numpy()[0]) * s0 + np.outer(x["v"][0, 0, -1].double(), x["k"][0, 0, -1].double())
    assert rel_err(st[0, 0], want, 0) <= TOL_F32


def test_scale_of_zero_and_of_other_sizes(B):
    for io, d in (("bf16", 128), ("f32", 32)):
        x = draw(1, 2, 1, 200, d, d, io, seed=11)
        for scale in (0.0, -3.0, 1e-3):
            check_fwd(B, x, scale=scale)
            check_bwd(B, x, scale=scale)


@pytest.mark.parametrize("kind", [(2, 2, 300, 128, 128, "bf16"), (2, 2, 300, 32, 32, "f32")], ids=str)
def test_bad_values_stay_within_their_head_and_sequence(B, kind):
    H, Hk, T, dk, dv, io = kind
    starts = [0, 100, 250, 290]
    x = draw(1, *kind, n=3, seed=12)
    x["v"][0, 0, 250 - 1, 3] = float("nan")
    x["k"][0, 0, 249, 5] = float("inf")
    x["q"][0, 0, 120, 5] = float("nan")
    for n in ("q", "k", "v", "dout"):
        x[n][0, :, 290:] = float("nan")  # behind the last sequence
    x["log_alpha"][0, :, 290:] = float("nan")
    o, st = gpu_fwd(B, x, starts)
    d = gpu_bwd(B, x, starts)
    clean = {n: t.clone() for n, t in x.items()}
    for n in ("q", "k", "v", "dout"):
        clean[n] = torch.nan_to_num(clean[n].float(), 0.0, 0.0, 0.0).to(clean[n].dtype)
    clean["log_alpha"] = torch.nan_to_num(clean["log_alpha"])
    oc, sc = gpu_fwd(B, clean, starts)
    dc = gpu_bwd(B, clean, starts)
    ok = np.ones((H, T), bool)
    ok[0, 100:250] = False
    assert np.array_equal(o[0][ok], oc[0][ok]) and np.array_equal(st[[0, 2]], sc[[0, 2]]) and np.array_equal(st[1, 1], sc[1, 1])
    for n, (a, c) in enumerate(zip(d[:4], dc[:4])):
        assert np.array_equal(a[0][ok], c[0][ok]), n
    assert np.isnan(o[0, 0, 249]).any()


def test_bad_starts_set_the_device_error(B):
    x = {n: t.to(DEV) for n, t in draw(1, 2, 1, 64, 32, 32, "f32", n=2, seed=3).items()}
    for starts in ([0, 40, 65], [5, 3, 64], [-1, 3, 64], [0, 64, 63]):
        ss = torch.tensor(starts, dtype=torch.int32, device=DEV)
        B.ll_la_fwd(x["q"], x["k"], x["v"], x["log_alpha"], state_in=x["state_in"], seq_starts=ss)
        assert B.ll_last_device_error() == 6, starts
        B.ll_la_bwd(x["q"], x["k"], x["v"], x["log_alpha"], x["dout"], seq_starts=ss)
        assert B.ll_last_device_error() == 6, starts


@pytest.mark.parametrize("kind", [(2, 1, 300, 128, 128, "bf16"), (4, 2, 333, 32, 64, "f32")], ids=str)
def test_repeats_are_equal_and_states_in_place(B, kind):
    x = draw(2, *kind, seed=4)
    g, st_shape, _, _ = setup(B, x, None, 0.5)
    a = (g["q"], g["k"], g["v"], g["log_alpha"])
    st = torch.empty(st_shape, device=DEV)
    o = B.ll_la_fwd(*a, state_in=g["state_in"], state_out=st)
    d = torch.empty(st_shape, device=DEV)
    grads = B.ll_la_bwd(*a, g["dout"], state_in=g["state_in"], dstate_out=g["dstate_out"], dstate_in=d)
    for _ in range(3):
        s2, d2 = g["state_in"].clone(), g["dstate_out"].clone()
        assert torch.equal(o, B.ll_la_fwd(*a, state_in=s2, state_out=s2)) and torch.equal(s2, st)
        again = B.ll_la_bwd(*a, g["dout"], state_in=g["state_in"], dstate_out=d2, dstate_in=d2)
        assert torch.equal(d2, d) and all(torch.equal(p, r) for p, r in zip(grads, again))
    assert B.ll_last_device_error() == 0


@pytest.mark.parametrize("kind", [(2, 1, 600, 128, 128, "bf16"), (2, 2, 200, 32, 32, "f32")], ids=str)
def test_captured_and_on_another_stream(B, kind):
    x, y = draw(1, *kind, seed=21), draw(1, *kind, seed=22)
    g, _, _, _ = setup(B, x, None, 0.5)
    a = (g["q"], g["k"], g["v"], g["log_alpha"])

    def both(g=g, a=a):
        return [B.ll_la_fwd(*a, state_in=g["state_in"]), *B.ll_la_bwd(*a, g["dout"], state_in=g["state_in"], dstate_out=g["dstate_out"])]

    want_x = [t.clone() for t in both()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    gy, _, _, _ = setup(B, y, None, 0.5)
    want_y = both(gy, (gy["q"], gy["k"], gy["v"], gy["log_alpha"]))
    for n in g:
        g[n].copy_(gy[n])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, r) for p, r in zip(other, want_x))
    assert all(torch.equal(p, r) for p, r in zip(out, want_y))


@pytest.mark.parametrize("kind", [(1, 1, 9001, 64, 64, "bf16"), (1, 1, 30001, 16, 16, "f32"), (2, 1, 5003, 128, 64, "bf16")], ids=str)
def test_many_segments(B, kind):
    """Long sequences of few heads, slow decays: states pass from segment to segment many times."""
    x = draw(1, *kind, seed=61, rate=1e-3)
    check_fwd(B, x)
    check_bwd(B, x)


@pytest.mark.parametrize("T", [15, 16, 17, 23, 24, 31, 32, 47, 48, 49, 63, 64])
@pytest.mark.parametrize("heads", [2, 154])
def test_short_sequences(B, heads, T):
    """Both sides of the lengths from which chunks are taken, with few states and with many."""
    for d in (64, 128):
        x = draw(1, heads, heads // 2, T, d, d, "bf16", seed=T, per_head=T % 2 == 0)
        check_fwd(B, x)
        if heads == 2:
            check_bwd(B, x)


@pytest.mark.parametrize("kind", [(2, 1, 300, 64, 128, "bf16"), (2, 1, 90, 32, 32, "f32")], ids=str)
def test_growth_is_computed_as_given(B, kind):
    x = draw(1, *kind, seed=62, init=False)
    x["log_alpha"] = x["log_alpha"].abs() * 0.02
    check_fwd(B, x)


@pytest.mark.parametrize("kind", [(2, 1, 500, 128, 64, "bf16"), (2, 2, 70, 32, 32, "f32")], ids=str)
def test_powers_of_two_pass_through(B, kind):
    """Products and sums of inputs times powers of two are those of the inputs, times powers of two: every bit."""
    x = draw(1, *kind, seed=68, init=False)
    e = dict(q=-30, k=45, v=25, dout=-28)
    y = dict(x, **{n: x[n] * 2.0 ** e[n] for n in e})
    (o, st), d = gpu_fwd(B, x), gpu_bwd(B, x)
    (oy, sty), dy = gpu_fwd(B, y), gpu_bwd(B, y)
    whole = sum(e.values())
    for a, b, by in [(o, oy, whole - e["dout"]), (st, sty, e["k"] + e["v"]), (d[0], dy[0], whole - e["q"]), (d[1], dy[1], whole - e["k"]),
                     (d[2], dy[2], whole - e["v"]), (d[3], dy[3], whole), (d[4], dy[4], e["q"] + e["dout"])]:
        assert np.array_equal(a * 2.0 ** by, b) and np.isfinite(b).all()


@pytest.mark.parametrize("kind", [(2, 2, 700, 128, 128, "bf16"), (2, 2, 700, 32, 32, "f32")], ids=str)
def test_bad_decays_stay_within_their_head_and_sequence(B, kind):
    starts, H, T = [0, 200, 650, 700], kind[0], kind[2]
    x = draw(1, *kind, n=3, seed=63)
    o0, s0 = gpu_fwd(B, x, starts)
    d0 = gpu_bwd(B, x, starts)
    x["log_alpha"][0, 1, 460] = float("nan")
    o, s = gpu_fwd(B, x, starts)
    d = gpu_bwd(B, x, starts)
    ok = np.ones((H, T), bool)
    ok[1, 200:650] = False
    assert np.array_equal(o[0][ok], o0[0][ok]) and np.array_equal(s[[0, 2]], s0[[0, 2]]) and np.array_equal(s[1, 0], s0[1, 0])
    for a, c in zip(d[:4], d0[:4]):
        assert np.array_equal(a[0][ok], c[0][ok])
    assert np.isnan(o[0, 1, 460:650]).all() and np.isnan(s[1, 1]).all() and np.array_equal(o[0, 1, 200:328], o0[0, 1, 200:328])
    assert np.isnan(d[3][0, 1, 200:461]).all() and np.isnan(d[4][1, 1]).all()


def test_two_graphs_at_once(B):
    """Two captured calls with workspaces of their own, replayed side by side on two streams."""
    kind = (4, 2, 2000, 128, 128, "bf16")
    xs = [setup(B, draw(1, *kind, seed=64 + i), None, 0.5)[0] for i in range(2)]

    def call(g):
        return [B.ll_la_fwd(g["q"], g["k"], g["v"], g["log_alpha"], state_in=g["state_in"]),
                *B.ll_la_bwd(g["q"], g["k"], g["v"], g["log_alpha"], g["dout"], dstate_out=g["dstate_out"])]

    want = [[t.clone() for t in call(g)] for g in xs]
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for g in xs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call(g))
    torch.cuda.synchronize()
    for _ in range(5):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(a, b) for a, b in zip(w, o))


TAIL, SHOWN = 900, 300  # of a sequence whose decays leave e^-300 of what lies before the tail


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_offsets_past_31_bits(B, io):
    """More elements than 31 bits count: the last tokens of the last head against the recurrence."""
    H, Hk, T, dk, dv = 8, 1, 2_200_000, 64, 128
    assert H * T * dv > 1 << 31
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    gen = torch.Generator(DEV).manual_seed(65)
    q, k, v, do = [torch.empty(1, h, T, d, dtype=dt, device=DEV).normal_(generator=gen)
                   for h, d in ((Hk, dk), (Hk, dk), (H, dv), (H, dv))]
    ga = torch.empty(1, H, T, device=DEV).uniform_(-0.6, -0.4, generator=gen)
    f = lambda x: x.double().cpu().numpy()
    tails = [[f(x[0, h if x.shape[1] == H else 0, -TAIL:]) for x in (q, k, v, ga, do)] for h in range(H)]
    tol = TOL_F32 if io == "f32" else TOL_BF16
    st = torch.empty(1, H, dv, dk, device=DEV)
    o = B.ll_la_fwd(q, k, v, ga, scale=0.5, state_out=st)
    ro, rs = la.forward(*tails[-1][:4], scale=0.5)
    assert rel_err(f(o[0, -1, -SHOWN:]), ro[-SHOWN:], 0) <= tol and rel_err(f(st[0, -1]), rs, 0) <= TOL_F32
    del o
    dq, dkey, dval, dla = B.ll_la_bwd(q, k, v, ga, do, scale=0.5)
    r = [la.backward(*t, scale=0.5) for t in tails]
    for got, name in ((dq, "dq"), (dkey, "dk")):
        assert rel_err(f(got[0, 0, -SHOWN:]), sum(x[name][-SHOWN:] for x in r), 0) <= tol, name
    assert rel_err(f(dval[0, -1, -SHOWN:]), r[-1]["dv"][-SHOWN:], 0) <= tol
    term = max(np.abs((tails[-1][0] * r[-1]["dq"]).sum(-1)).max(), r[-1]["terms"].max())
    assert np.abs(f(dla[0, -1, -SHOWN:]) - r[-1]["dlog_alpha"][-SHOWN:]).max() <= TOL_F32 * term
    assert B.ll_last_device_error() == 0


def test_gradient_against_differences(B):
    """float32, token by token: a directional derivative of sum(o . dout) + sum(S . dS) computed in 64 bits."""
    x = draw(1, 2, 1, 90, 32, 16, "f32", seed=31)
    got = gpu_bwd(B, x)
    r = np.random.default_rng(0)
    names = ("q", "k", "v", "log_alpha", "state_in")
    f = {n: t.double().numpy() for n, t in x.items()}
    step = {n: r.standard_normal(f[n].shape) for n in names}

    def loss(e):
        z = {n: torch.from_numpy(f[n] + e * step[n]) if n in step else x[n].double() for n in f}
        tot = 0.0
        for _, a, do, s0, ds in slices(z, None):
            o, s = la.forward(*a, scale=0.5, state=s0)
            tot += (o * do).sum() + (s * ds).sum()
        return tot

    want = (loss(1e-5) - loss(-1e-5)) / 2e-5
    have = sum((g.astype(np.float64) * step[n]).sum() for g, n in zip(got, names))
    size = np.sqrt(sum(((g.astype(np.float64) * step[n]) ** 2).sum() for g, n in zip(got, names)))
    assert abs(have - want) <= 1e-4 * size


# ---------------------------------------------------------------- one token
STEPS = [(1, 1, 1, 16, 16, "f32"), (3, 4, 2, 32, 64, "bf16"), (2, 2, 2, 64, 16, "f32"), (5, 4, 1, 128, 128, "bf16"),
         (2, 2, 1, 16, 128, "bf16"), (1, 32, 16, 128, 128, "f32"), (4, 2, 1, 128, 32, "bf16"), (2, 3, 3, 64, 64, "bf16")]


@pytest.mark.parametrize("rope", [None, (1.0, False), (0.5, True), (0.3, False)], ids=str)
@pytest.mark.parametrize("kind", STEPS, ids=str)
def test_step(B, kind, rope):
    Bn, H, Hk, dk, dv, io = kind
    for per_head in (False, True):
        x = draw(Bn, H, Hk, 1, dk, dv, io, seed=41, per_head=per_head)
        pool = Bn + 3
        states = torch.randn(pool, H, dv, dk, generator=torch.Generator().manual_seed(2))
        slots = torch.randperm(pool, generator=torch.Generator().manual_seed(3))[:Bn]
        if Bn > 1:
            slots[1] = -1
        g = {n: t.to(DEV) for n, t in x.items()}
        st, o = Guarded(states.shape, torch.float32, fill=states), Guarded((Bn, H, dv), g["q"].dtype, fill=SEVEN)
        more, f = {}, None
        if rope:
            rot = max(2, int(rope[0] * dk) // 2 * 2)
            f = B.ll_rope_freqs(rot)
            pos = torch.tensor([3, 70000, 0, 5, 1 << 20][:Bn])
            more = dict(inv_freq=f.to(DEV), positions=pos.to(DEV), interleaved=rope[1], amp=1.25)
        la_in = g["log_alpha"] if per_head else g["log_alpha"][:, :, 0].contiguous()
        B.ll_la_decode_step(*[g[n][:, :, 0].contiguous() for n in ("q", "k", "v")], la_in, st.view, scale=0.5, slots=slots.to(DEV),
                            o=o.view, **more)
        assert B.ll_last_device_error() == 0 and st.intact() and o.intact()
        want, wo = states.double().numpy().copy(), np.full((Bn, H, dv), 7.0)
        d = {n: t.double().numpy() for n, t in x.items()}
        if rope:
            for n in ("q", "k"):
                d[n] = la.rope(d[n], pos.numpy()[:, None, None], f.numpy(), rope[1], 1.25)
        for b in range(Bn):
            for h in range(H):
                if slots[b] >= 0:
                    ga = d["log_alpha"][h:h + 1] if per_head else d["log_alpha"][b, h]
                    oo, want[slots[b], h] = la.forward(d["q"][b, h // (H // Hk)], d["k"][b, h // (H // Hk)], d["v"][b, h], ga,
                                                       0.5, want[slots[b], h])
                    wo[b, h] = oo[0]
        assert rel_err(st.view.cpu().numpy(), want) <= TOL_F32
        assert rel_err(o.view.float().cpu().numpy(), wo) <= (TOL_F32 if io == "f32" else 2.0 ** -8 + TOL_F32)
        if Bn > 1:
            assert (o.view[1] == 7).all()


def test_step_forgets_whatever_a_slot_holds(B):
    x = {n: t.to(DEV)[:, :, 0].contiguous() for n, t in draw(2, 2, 1, 1, 64, 64, "bf16", seed=5, init=False).items()}
    st = torch.full((2, 2, 64, 64), float("nan"), device=DEV)
    x["log_alpha"][:] = -float("inf")
    o = B.ll_la_decode_step(x["q"], x["k"], x["v"], x["log_alpha"], st)
    want = x["v"].float()[..., None] * x["k"].float()[:, :, None, :]
    assert torch.equal(st, want.expand_as(st)) and torch.isfinite(o).all()


def test_step_bad_slots(B):
    x = {n: t.to(DEV)[:, :, 0].contiguous() for n, t in draw(3, 2, 1, 1, 32, 32, "f32", seed=5, init=False).items()}
    for slots in ([0, 4, 1], [0, -2, 1], [2, 1, 2]):
        st = torch.zeros(4, 2, 32, 32, device=DEV)
        B.ll_la_decode_step(x["q"], x["k"], x["v"], x["log_alpha"], st, slots=torch.tensor(slots, device=DEV))
        assert B.ll_last_device_error() == 6, slots
    assert B.ll_last_device_error() == 0


def test_step_states_past_31_bits(B):
    """A pool of more elements than 31 bits count, its last slots."""
    H, d, n = 32, 128, 4200
    assert n * H * d * d > 1 << 31
    x = draw(3, H, H, 1, d, d, "f32", seed=66, init=False)
    g = {m: t.to(DEV)[:, :, 0].contiguous() for m, t in x.items()}
    pool = torch.empty(n, H, d, d, device=DEV)
    slots = [n - 1, 1, n - 2]
    start = torch.randn(3, H, d, d, generator=torch.Generator().manual_seed(1))
    pool[-4:] = 7.0
    pool[torch.tensor(slots, device=DEV)] = start.to(DEV)
    o = B.ll_la_decode_step(g["q"], g["k"], g["v"], g["log_alpha"], pool, slots=torch.tensor(slots, device=DEV)).cpu().numpy()
    for (i, b, h, *_), a, _, _, _ in slices(x, None):
        ro, rs = la.forward(*a, state=start[b, h].double().numpy())
        assert rel_err(o[b, h], ro[0], 0) <= TOL_F32 and rel_err(pool[slots[b], h].cpu().numpy(), rs, 0) <= TOL_F32
    assert (pool[-4:-2] == 7).all() and B.ll_last_device_error() == 0


# ---------------------------------------------------------------- rotary positions
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("kind", [(1, 1, 1, 1, 16, 2, "f32"), (2, 4, 2, 5, 64, 64, "bf16"), (1, 16, 3, 33, 128, 96, "bf16"),
                                  (3, 2, 0, 7, 32, 20, "f32"), (1, 9, 9, 130, 128, 128, "f32"), (2, 5, 1, 3, 64, 6, "bf16"),
                                  (1, 40, 8, 17, 16, 16, "bf16")], ids=str)
def test_rope(B, kind, inter):
    Bn, H, Hk, T, d, rot, io = kind
    g = torch.Generator().manual_seed(1)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    q = torch.randn(Bn, H, T, d, generator=g).to(dt)
    k = torch.randn(Bn, Hk, T, d, generator=g).to(dt) if Hk else None
    f = B.ll_rope_freqs(rot, 10000.0)
    tol = TOL_F32 if io == "f32" else 2.0 ** -8 + TOL_F32
    far = torch.randint(-5, 1 << 22, (Bn, T), generator=g)
    for pos in (None, far):
        for back in (False, True):
            call = B.ll_rope_bwd if back else B.ll_rope_fwd
            gq, gk = Guarded(q.shape, dt, fill=SEVEN), Guarded(k.shape, dt, fill=SEVEN) if Hk else None
            names = ("dq", "dk") if back else ("q_out", "k_out")
            outs = {names[0]: gq.view, **({names[1]: gk.view} if Hk else {})}
            call(q.to(DEV), k.to(DEV) if Hk else None, f.to(DEV), positions=None if pos is None else pos.to(DEV), interleaved=inter, amp=0.7, **outs)
            at = (np.arange(T)[None] if pos is None else pos.numpy())[:, None]
            for x, y in ((q, gq), (k, gk)):
                if x is None:
                    continue
                assert y.intact()
                want = la.rope(x.double().numpy(), at, f.numpy(), inter, 0.7, back)
                # a rotation's error is that of its pair's size
                assert np.abs(y.view.double().cpu().numpy() - want).max() <= tol * np.abs(want).max()
                assert torch.equal(y.view[..., rot:].cpu(), x[..., rot:])
            inq, ink = q.to(DEV), k.to(DEV) if Hk else None
            call(inq, ink, f.to(DEV), positions=None if pos is None else pos.to(DEV), interleaved=inter, amp=0.7,
                 **{names[0]: inq, **({names[1]: ink} if Hk else {})})
            assert torch.equal(inq, gq.view) and (not Hk or torch.equal(ink, gk.view))


def test_rope_angles_at_far_positions(B):
    """cos and sin themselves, float32: off by no more than the fixed-point angle (2^-31 of a half turn,
    1.5e-9 radians) and the rounding of both, 3 x 2^-24, whatever the position."""
    f = torch.cat([B.ll_rope_freqs(60), torch.tensor([1.9, 2.5])])
    pos = torch.tensor([[0, 1, -1, 1000003, (1 << 31) - 1, 1 << 31, -(1 << 33) + 5, (1 << 40) - 1]])
    x = torch.zeros(1, 1, 8, 64)
    x[..., :32] = 1.0
    got = B.ll_rope_fwd(x.to(DEV), None, f.to(DEV), positions=pos.to(DEV)).double().cpu().numpy()
    want = la.rope(x.numpy(), pos.numpy()[:, None], f.numpy())
    assert np.abs(got - want)[:, :, :5].max() <= 2e-9 + 3 * 2.0 ** -24
    assert np.abs(got - want).max() <= 2e-9 + 3 * 2.0 ** -24 + 2 * np.pi * 2.0 ** -22  # (2^40 positions, 2^-64 + 2^-63 of a turn each)


def test_rope_offsets_past_31_bits(B):
    H, Hk, T, d = 9, 8, 2_000_000, 128
    assert H * T * d > 1 << 31
    gen = torch.Generator(DEV).manual_seed(67)
    q, k = [torch.empty(1, h, T, d, dtype=torch.bfloat16, device=DEV).normal_(generator=gen) for h in (H, Hk)]
    tail = [t[0, -1, -50:].double().cpu().numpy() for t in (q, k)]
    f = B.ll_rope_freqs(d)
    B.ll_rope_fwd(q, k, f.to(DEV), q_out=q, k_out=k)
    for t, w in zip((q, k), tail):
        want = la.rope(w, np.arange(T - 50, T), f.numpy())
        assert rel_err(t[0, -1, -50:].double().cpu().numpy(), want) <= 2.0 ** -8 + TOL_F32


def test_rope_of_single_tokens(B):
    q, k = torch.randn(3, 4, 64, device=DEV), torch.randn(3, 2, 64, device=DEV)
    f, pos = B.ll_rope_freqs(64, device=DEV), torch.tensor([4, 0, 99], device=DEV)
    a, b = B.ll_rope_fwd(q, k, f, positions=pos)
    c, d = B.ll_rope_fwd(q[:, :, None].contiguous(), k[:, :, None].contiguous(), f, positions=pos[:, None].contiguous())
    assert torch.equal(a, c[:, :, 0]) and torch.equal(b, d[:, :, 0])
    with pytest.raises(ValueError):
        B.ll_rope_fwd(q, k, f)


# ---------------------------------------------------------------- together
def test_prompt_then_tokens(B):
    """Positions, a prompt, then tokens one by one against the whole sequence in 64 bits."""
    Bn, H, Hk, T, n, d = 2, 4, 2, 200, 6, 64
    x = draw(Bn, H, Hk, T + n, d, d, "f32", seed=51, init=False, per_head=True)
    f = B.ll_rope_freqs(48, factor=4.0, length=128.0)
    g = {m: t.to(DEV) for m, t in x.items()}
    fd = f.to(DEV)
    q, k = B.ll_rope_fwd(g["q"][:, :, :T].contiguous(), g["k"][:, :, :T].contiguous(), fd)
    st = torch.empty(Bn, H, d, d, device=DEV)
    o = [B.ll_la_fwd(q, k, g["v"][:, :, :T].contiguous(), g["log_alpha"], scale=0.1, state_out=st)]
    pool, slots = torch.zeros(5, H, d, d, device=DEV), torch.tensor([3, 1], device=DEV)
    pool[slots] = st
    for t in range(T, T + n):
        o.append(B.ll_la_decode_step(*[g[m][:, :, t].contiguous() for m in ("q", "k", "v")], g["log_alpha"], pool, scale=0.1, slots=slots,
                                     inv_freq=fd, positions=torch.full((Bn,), t, device=DEV))[:, :, None])
    o = torch.cat(o, 2).cpu().numpy()
    y = dict(x, **{m: torch.from_numpy(la.rope(x[m].double().numpy(), np.arange(T + n), f.numpy())) for m in ("q", "k")})
    for (i, b, h, *_), a, _, _, _ in slices(y, None):
        ro, rs = la.forward(*a, scale=0.1)
        assert rel_err(o[b, h], ro, 0) <= TOL_F32
        assert rel_err(pool[slots[b], h].cpu().numpy(), rs, 0) <= TOL_F32
    assert (pool[[0, 2, 4]] == 0).all() and B.ll_last_device_error() == 0


def test_training_step_through_positions(B):
    """The gradients of unturned queries and keys, bf16: turned, attended, back, turned back."""
    Bn, H, Hk, T, d = 1, 2, 1, 300, 64
    x = draw(Bn, H, Hk, T, d, d, "bf16", seed=52, init=False)
    f = B.ll_rope_freqs(d)
    g = {m: t.to(DEV) for m, t in x.items()}
    q, k = B.ll_rope_fwd(g["q"], g["k"], f.to(DEV))
    dq, dk, dv, dla = B.ll_la_bwd(q, k, g["v"], g["log_alpha"], g["dout"], scale=0.125)
    dq, dk = B.ll_rope_bwd(dq, dk, f.to(DEV))
    y = dict(x, **{m: torch.from_numpy(la.rope(x[m].double().numpy(), np.arange(T), f.numpy())) for m in ("q", "k")})
    want = {m: np.zeros((T, d)) for m in ("dq", "dk")}
    for (i, b, h, *_), a, do, _, _ in slices(y, None):
        r = la.backward(*a, do, scale=0.125)
        for m in want:
            want[m] += la.rope(r[m], np.arange(T), f.numpy(), back=True)
        assert rel_err(dv[b, h].float().cpu().numpy(), r["dv"], 0) <= TOL_BF16
    for m, got in (("dq", dq), ("dk", dk)):
        assert rel_err(got[0, 0].float().cpu().numpy(), want[m], 0) <= TOL_BF16
