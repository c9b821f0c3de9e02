"""GPU parity of the gated delta rule (ll_gdr_fwd, ll_gdr_bwd,
ll_gdr_decode_step) against the recurrence in 64 bits (oracle.gdr).

Tolerances, relative to a (sequence, head) slice's largest value.  float32
values: TOL_F32, as every float32 path here (rounding of float32 sums).  bf16
outputs of float32 arithmetic (the token-by-token path, the decode step): half a
step of bf16, 2^-8, on top of that.  bf16 outputs of the tensor-core path, whose
operands (states, written rows, masked scores) are rounded to 16 bits once each:
TOL_BF16, as every bf16 tensor-core path here."""

import numpy as np
import pytest
import torch

from oracle import gdr
from tests._parity import TOL_BF16, TOL_F32, Guarded, rel_err

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def B():
    from log_linear_attention_chunked_gb300 import binding
    binding.lib()
    return binding


def draw(Bn, H, Hk, T, dk, dv, io="bf16", n=None, seed=0, init=True, slow=True):
    """CPU tensors of one call; n: states (sequences)."""
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32

    def r(*s):
        return torch.randn(*s, generator=g)

    def unit(x):
        return torch.nn.functional.normalize(torch.nn.functional.silu(x), dim=-1).to(dt)

    rate = torch.logspace(-2.7, -0.2, H).view(1, H, 1) if slow else torch.ones(1, H, 1)
    x = dict(q=unit(r(Bn, Hk, T, dk)), k=unit(r(Bn, Hk, T, dk)), v=r(Bn, H, T, dv).to(dt),
             log_alpha=-rate * torch.nn.functional.softplus(r(Bn, H, T)), beta=torch.sigmoid(r(Bn, H, T)),
             dout=r(Bn, H, T, dv).to(dt))
    if init:
        x["state_in"] = 0.3 * r(n or Bn, H, dv, dk)
        x["dstate_out"] = 0.3 * r(n or Bn, H, dv, dk)
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
            a = [f["q"][b, hk, lo:hi], f["k"][b, hk, lo:hi], *[f[n][b, h, lo:hi] for n in ("v", "log_alpha", "beta")]]
            st = f["state_in"][i, h] if "state_in" in f else None
            ds = f["dstate_out"][i, h] if "dstate_out" in f else None
            yield (i, b, h, hk, lo, hi), a, f["dout"][b, h, lo:hi], st, ds


def gpu_fwd(B, x, starts=None, scale=0.5, guard=True):
    g = {n: t.to(DEV) for n, t in x.items()}
    Bn, Hk, T, dk = g["q"].shape
    _, H, _, dv = g["v"].shape
    n = Bn if starts is None else len(starts) - 1
    o, st = Guarded(tuple(g["v"].shape), g["v"].dtype, fill=torch.tensor(7.0)), Guarded((n, H, dv, dk), torch.float32)
    shape = B.make_gdr_shape(Bn, H, Hk, T, dk, dv, 0 if starts is None else n, scale, B._io(g["q"].dtype))
    ws = Guarded((max(256, B.ll_gdr_fwd_workspace_size(shape)),), torch.uint8)
    ss = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)
    B.ll_gdr_fwd(g["q"], g["k"], g["v"], g["log_alpha"], g["beta"], scale=scale, state_in=g.get("state_in"),
                 state_out=st.view, seq_starts=ss, o=o.view, workspace=ws.view)
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
        ro, rs = gdr.forward(*a, scale=scale, state=s0)
        covered[b, h, lo:hi] = True
        assert rel_err(st[i, h], rs, 0) <= TOL_F32, (i, h, "state")
        if hi > lo:
            assert rel_err(o[b, h, lo:hi], ro, 0) <= tol_out(x), (i, h, "o")
    assert (o[~covered] == 7.0).all(), "a row outside every sequence was written"


def gpu_bwd(B, x, starts=None, scale=0.5):
    g = {n: t.to(DEV) for n, t in x.items()}
    Bn, Hk, T, dk = g["q"].shape
    _, H, _, dv = g["v"].shape
    n = Bn if starts is None else len(starts) - 1
    io = g["q"].dtype
    seven = torch.tensor(7.0)
    out = [Guarded(tuple(g[s].shape), g[s].dtype, fill=seven) for s in ("q", "k", "v", "log_alpha", "beta")]
    ds = Guarded((n, H, dv, dk), torch.float32)
    shape = B.make_gdr_shape(Bn, H, Hk, T, dk, dv, 0 if starts is None else n, scale, B._io(io))
    ws = Guarded((B.ll_gdr_bwd_workspace_size(shape),), torch.uint8)
    ss = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)
    B.ll_gdr_bwd(g["q"], g["k"], g["v"], g["log_alpha"], g["beta"], g["dout"], scale=scale,
                 state_in=g.get("state_in"), dstate_out=g.get("dstate_out"), seq_starts=ss,
                 grads=[t.view for t in out], dstate_in=ds.view, workspace=ws.view)
    assert B.ll_last_device_error() == 0
    assert all(t.intact() for t in out) and ds.intact() and ws.intact(), "write outside a buffer"
    return [t.view.float().cpu().numpy() for t in out] + [ds.view.cpu().numpy()]


def check_bwd(B, x, starts=None, scale=0.5):
    dq, dk, dv, dla, db, dst = gpu_bwd(B, x, starts, scale)
    rq, rk = np.full(dq.shape, 7.0), np.full(dk.shape, 7.0)
    covered = np.zeros(dv.shape[:3], bool)
    for i, b, lo, hi in seqs_of(x, starts):
        rq[b, :, lo:hi] = rk[b, :, lo:hi] = 0.0
    for (i, b, h, hk, lo, hi), a, do, s0, ds in slices(x, starts):
        r = gdr.backward(*a, do, scale=scale, state=s0, dstate=ds)
        assert rel_err(dst[i, h], r["dstate_in"], 0) <= TOL_F32, (i, h, "dstate_in")
        covered[b, h, lo:hi] = True
        if hi == lo:
            continue
        rq[b, hk, lo:hi] += r["dq"]
        rk[b, hk, lo:hi] += r["dk"]
        assert rel_err(dv[b, h, lo:hi], r["dv"], 0) <= tol_out(x), (i, h, "dv")
        # the gates' gradients are sums of do.o, v.dv and e.w, which may cancel:
        # their rounding is relative to those terms (reading R12b)
        o, _ = gdr.forward(*a, scale=scale, state=s0)
        terms = max(np.abs((do * o).sum(-1)).max(), np.abs((a[2] * r["dv"]).sum(-1)).max())
        for name, got in (("dlog_alpha", dla), ("dbeta", db)):
            # (1e-30 as in rel_err: a gradient of 1e-64, a decay of e^-144 through a sequence without
            # inputs, has no float32 next to it, whose smallest value is 2^-149 = 1.4e-45)
            den = max(np.abs(r[name]).max(), terms, 1e-30)
            assert np.abs(got[b, h, lo:hi] - r[name]).max() <= TOL_F32 * den, (i, h, name)
    for name, got, ref in (("dq", dq, rq), ("dk", dk, rk)):
        for i, b, lo, hi in seqs_of(x, starts):
            if hi > lo:
                assert rel_err(got[b, :, lo:hi], ref[b, :, lo:hi], 1) <= tol_out(x), (i, name)
    assert (dv[~covered] == 7.0).all() and (dla[~covered] == 7.0).all() and (db[~covered] == 7.0).all()
    Hk, H = dq.shape[1], dv.shape[1]
    un = ~covered[:, ::H // Hk]
    assert (dq[un] == 7.0).all() and (dk[un] == 7.0).all(), "a row outside every sequence was written"


SHAPES = [  # B, H, Hk, T, dk, dv, io
    (1, 1, 1, 1, 16, 16, "f32"), (2, 2, 1, 2, 32, 16, "f32"), (1, 2, 2, 15, 16, 32, "bf16"),
    (1, 4, 2, 16, 64, 64, "bf16"), (1, 3, 1, 17, 128, 128, "f32"), (2, 2, 2, 63, 64, 128, "bf16"),
    (1, 2, 1, 64, 128, 64, "bf16"), (1, 4, 1, 65, 32, 32, "f32"), (3, 2, 1, 130, 16, 128, "f32"),
    (1, 2, 2, 333, 64, 32, "f32"),
    # bf16 with head sizes of 64 and 128, where long ones run on the tensor cores
    (1, 2, 1, 400, 64, 128, "bf16"), (2, 2, 2, 260, 128, 64, "bf16"), (1, 3, 3, 512, 64, 64, "bf16"),
    (1, 1, 1, 1, 128, 128, "bf16"), (2, 2, 1, 31, 128, 128, "bf16"), (1, 2, 2, 127, 128, 128, "bf16"),
    (1, 2, 1, 128, 128, 128, "bf16"), (2, 4, 2, 129, 128, 128, "bf16"), (1, 2, 2, 511, 128, 128, "bf16"),
    (1, 2, 1, 1000, 128, 128, "bf16"), (1, 2, 2, 1024, 128, 128, "bf16"),
]


@pytest.mark.parametrize("init", [True, False])
@pytest.mark.parametrize("Bn,H,Hk,T,dk,dv,io", SHAPES)
def test_forward_shapes(B, Bn, H, Hk, T, dk, dv, io, init):
    check_fwd(B, draw(Bn, H, Hk, T, dk, dv, io, seed=T, init=init))


@pytest.mark.parametrize("init", [True, False])
@pytest.mark.parametrize("Bn,H,Hk,T,dk,dv,io", SHAPES)
def test_backward_shapes(B, Bn, H, Hk, T, dk, dv, io, init):
    check_bwd(B, draw(Bn, H, Hk, T, dk, dv, io, seed=T, init=init))


# packed: empty sequences at both ends and in the middle, single tokens, ends
# inside and on a chunk's border, tokens before the first and behind the last
PACKED = [[0, 5], [0, 0, 1, 1, 20, 20], [3, 3, 66, 67, 131, 131, 259, 300, 300], [0, 128, 256, 257, 640, 641],
          [10, 138, 150], [0, 700]]
SETS = [(2, 1, 32, 16, "f32"), (2, 2, 64, 64, "bf16"), (4, 2, 128, 128, "bf16"), (2, 1, 128, 128, "f32")]


@pytest.mark.parametrize("H,Hk,dk,dv,io", SETS)
@pytest.mark.parametrize("starts", PACKED)
def test_packed(B, starts, H, Hk, dk, dv, io):
    x = draw(1, H, Hk, starts[-1] + 9, dk, dv, io, n=len(starts) - 1, seed=len(starts))
    # what lies outside every sequence must not matter
    for n in ("q", "k", "v", "log_alpha", "beta", "dout"):
        x[n][:, :, starts[-1]:] = float("nan")
        x[n][:, :, :starts[0]] = float("nan")
    check_fwd(B, x, starts)
    check_bwd(B, x, starts)


@pytest.mark.parametrize("dk,io", [(128, "bf16"), (32, "f32")])
def test_a_sequence_of_nan_stays_alone(B, dk, io):
    starts = [0, 100, 333, 400, 650]
    x = draw(1, 2, 1, 650, dk, dk, io, n=4, seed=8)
    ref_o, ref_s = gpu_fwd(B, x, starts)
    ref_g = gpu_bwd(B, x, starts)
    for n in ("q", "k", "v", "dout", "log_alpha", "beta"):
        x[n][:, :, 100:333] = float("nan")
    o, s = gpu_fwd(B, x, starts)
    g = gpu_bwd(B, x, starts)
    keep = np.r_[0:100, 333:650]
    assert np.array_equal(o[:, :, keep], ref_o[:, :, keep])
    assert np.array_equal(s[[0, 2, 3]], ref_s[[0, 2, 3]]) and np.isnan(s[1]).any()
    for a, b in zip(g[:5], ref_g[:5]):
        assert np.array_equal(a[:, :, keep], b[:, :, keep])
    assert np.array_equal(g[5][[0, 2, 3]], ref_g[5][[0, 2, 3]])


@pytest.mark.parametrize("dk,io,T", [(128, "bf16", 700), (64, "f32", 300)])
@pytest.mark.parametrize("what", ["forget", "no_write", "full_write", "no_decay", "strong", "zero_keys"])
def test_gates_at_their_limits(B, dk, io, T, what):
    x = draw(1, 2, 1, T, dk, dk, io, seed=11)
    if what == "forget":      # alpha = 0: the state is dropped
        x["log_alpha"][:, :, [0, 1, 50, 127, 128, 255, T - 1]] = -float("inf")
    elif what == "no_write":  # beta = 0, as in padding
        x["beta"][:, :, 20:200] = 0.0
    elif what == "full_write":
        x["beta"][:] = 1.0
    elif what == "no_decay":
        x["log_alpha"][:] = 0.0
    elif what == "strong":
        x["log_alpha"] = 40 * x["log_alpha"] - 3
    else:
        x["k"][:, :, ::3] = 0
    check_fwd(B, x)
    check_bwd(B, x)


def test_decay_near_one_in_chunks(B):
    """alpha = 0.9999 and faint writes: a state is scaled by thousands of decays, whose
    errors must not lean to one side."""
    x = draw(1, 2, 1, 3000, 128, 128, seed=32)
    x["log_alpha"][:] = -1e-4
    x["beta"] *= 0.02
    check_fwd(B, x)
    check_bwd(B, x)


def test_padding_after_a_prompt_changes_nothing(B):
    """beta = 0 and log_alpha = 0 behind the real tokens: the state stays."""
    x = draw(2, 2, 2, 300, 128, 128, "bf16", seed=12)
    x["beta"][:, :, 211:] = 0.0
    x["log_alpha"][:, :, 211:] = 0.0
    o, s = gpu_fwd(B, x)
    y = {n: t[:, :, :211].contiguous() if t.shape[2] == 300 else t for n, t in x.items()}
    for (i, b, h, hk, lo, hi), a, _, s0, _ in slices(y, None):
        assert rel_err(s[i, h], gdr.forward(*a, scale=0.5, state=s0)[1], 0) <= TOL_F32


@pytest.mark.parametrize("T", [40, 600])
def test_state_in_place(B, T):
    x = {n: t.to(DEV) for n, t in draw(2, 2, 1, T, 128, 128, "bf16", seed=13).items()}
    args = [x[n] for n in ("q", "k", "v", "log_alpha", "beta")]
    out = torch.empty_like(x["state_in"])
    o = B.ll_gdr_fwd(*args, state_in=x["state_in"], state_out=out)
    st = x["state_in"].clone()
    o2 = B.ll_gdr_fwd(*args, state_in=st, state_out=st)
    assert torch.equal(o, o2) and torch.equal(st, out)
    ds = torch.empty_like(out)
    g = B.ll_gdr_bwd(*args, x["dout"], state_in=x["state_in"], dstate_out=x["dstate_out"], dstate_in=ds)
    d2 = x["dstate_out"].clone()
    g2 = B.ll_gdr_bwd(*args, x["dout"], state_in=x["state_in"], dstate_out=d2, dstate_in=d2)
    assert torch.equal(ds, d2) and all(torch.equal(a, b) for a, b in zip(g, g2))


def test_pieces_equal_the_whole(B):
    """A prompt in pieces through the states, then token by token: as used in serving."""
    T, H, Hk = 420, 4, 2
    x = {n: t.to(DEV) for n, t in draw(1, H, Hk, T, 128, 128, "bf16", seed=14, init=False).items()}
    args = [x[n] for n in ("q", "k", "v", "log_alpha", "beta")]
    whole = torch.empty(1, H, 128, 128, device=DEV)
    o = B.ll_gdr_fwd(*args, scale=0.5, state_out=whole)
    st, outs = torch.zeros(1, H, 128, 128, device=DEV), []
    for lo, hi in ((0, 300), (300, 301), (301, 400)):
        outs.append(B.ll_gdr_fwd(*[t[:, :, lo:hi].contiguous() for t in args], scale=0.5, state_in=st, state_out=st))
    pool = torch.full((3, H, 128, 128), 5.0, device=DEV)
    pool[2] = st[0]
    slot = torch.tensor([2], device=DEV)
    for t in range(400, T):
        one = [a[:, :, t].contiguous() for a in args]
        outs.append(B.ll_gdr_decode_step(*one, pool, scale=0.5, slots=slot)[:, :, None])
    assert B.ll_last_device_error() == 0
    assert rel_err(pool[2].cpu().numpy(), whole[0].cpu().numpy(), 1) <= 2 * TOL_F32
    # each side within TOL_BF16 of the exact values
    assert rel_err(torch.cat(outs, 2).float().cpu().numpy(), o.float().cpu().numpy()) <= 2 * TOL_BF16
    assert (pool[:2] == 5.0).all()


def test_training_step_shifts_the_loss(B):
    """The gradient of all inputs at once predicts the change of f = sum(o . dout):
    f(x + h g) - f(x - h g) = 2 h |g|^2 + O(h^3), in float32."""
    x = {n: t.to(DEV) for n, t in draw(1, 2, 1, 200, 32, 32, "f32", seed=15, init=False).items()}
    names = ("q", "k", "v", "log_alpha", "beta")
    g = B.ll_gdr_bwd(*[x[n] for n in names], x["dout"])
    sq = sum(float(t.double().square().sum()) for t in g)

    def f(h):
        moved = [(x[n] + h * t).contiguous() for n, t in zip(names, g)]
        return float((B.ll_gdr_fwd(*moved).double() * x["dout"].double()).sum())

    h = 1e-3 / sq ** 0.5
    # h |g| = 1e-3: the cubic term is 1e-6 of the linear one times the ratio of third to first
    # derivatives (order 1-10 here); float32 rounding of f (1e-7 |f|) over 2 h |g|^2 is below 1e-3
    got = (f(h) - f(-h)) / (2 * h)
    assert abs(got - sq) <= 5e-3 * sq


@pytest.mark.parametrize("T", [50, 500])
def test_streams_and_graphs(B, T):
    """On a side stream, and captured: one graph for the forward, one for the
    backward, each with its own workspace, replayed in turn after new inputs."""
    mk = lambda seed: {n: t.to(DEV) for n, t in draw(1, 4, 2, T, 128, 128, "bf16", seed=seed).items()}  # noqa: E731
    names = ("q", "k", "v", "log_alpha", "beta")
    x, y = mk(16), mk(17)

    def both(x):
        st, ds = torch.empty_like(x["state_in"]), torch.empty_like(x["state_in"])
        o = B.ll_gdr_fwd(*[x[n] for n in names], state_in=x["state_in"], state_out=st)
        g = B.ll_gdr_bwd(*[x[n] for n in names], x["dout"], state_in=x["state_in"], dstate_out=x["dstate_out"],
                         dstate_in=ds)
        return [o, st, *g, ds]

    want_x, want_y = both(x), both(y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = both(x)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want_x))
    buf = {n: t.clone() for n, t in x.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(buf)
    for src, want in ((y, want_y), (x, want_x), (y, want_y)):
        for n in buf:
            buf[n].copy_(src[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert B.ll_last_device_error() == 0


@pytest.mark.parametrize("starts", [[0, 50, 30, 200], [-1, 20], [0, 201], [0, 5, 1 << 30, 7], [200, 0],
                                    [0, 200, 0, 200, 0, 200]])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_bad_starts_are_reported(B, starts, io):
    n = len(starts) - 1
    x = draw(1, 2, 1, 200, 128, 128, io, n=n, seed=18)
    g = {m: t.to(DEV) for m, t in x.items()}
    ss = torch.tensor(starts, dtype=torch.int32, device=DEV)
    args = [g[m] for m in ("q", "k", "v", "log_alpha", "beta")]
    shape = B.make_gdr_shape(1, 2, 1, 200, 128, 128, n, 1.0, B._io(g["q"].dtype))
    o, st = Guarded((1, 2, 200, 128), g["v"].dtype), Guarded((n, 2, 128, 128), torch.float32)
    ws = Guarded((max(256, B.ll_gdr_fwd_workspace_size(shape)),), torch.uint8)
    B.ll_gdr_fwd(*args, state_in=g["state_in"], state_out=st.view, seq_starts=ss, o=o.view, workspace=ws.view)
    assert B.ll_last_device_error() == 6
    assert o.intact() and st.intact() and ws.intact()
    ws = Guarded((B.ll_gdr_bwd_workspace_size(shape),), torch.uint8)
    out = [Guarded(tuple(t.shape), t.dtype) for t in args]
    B.ll_gdr_bwd(*args, g["dout"], state_in=g["state_in"], seq_starts=ss, grads=[t.view for t in out],
                 workspace=ws.view)
    assert B.ll_last_device_error() == 6
    assert all(t.intact() for t in out) and ws.intact()
    check_fwd(B, x, [0, 10, 200] if n == 2 else [0] * n + [200])  # and the next call is right again


# ------------------------------------------------------------------ the decode step
@pytest.mark.parametrize("Bn,H,Hk,dk,dv,io,pool", [
    (1, 1, 1, 16, 16, "f32", None), (3, 2, 1, 32, 64, "bf16", 7), (5, 4, 4, 64, 16, "f32", 5),
    (2, 32, 16, 128, 128, "bf16", None), (130, 2, 1, 128, 128, "bf16", 150), (7, 6, 2, 128, 32, "f32", 9),
    (2, 2, 2, 64, 128, "bf16", None)])
def test_decode_step(B, Bn, H, Hk, dk, dv, io, pool):
    x = draw(Bn, H, Hk, 1, dk, dv, io, seed=19)
    g = torch.Generator().manual_seed(3)
    n = pool or Bn
    states = 0.5 * torch.randn(n, H, dv, dk, generator=g)
    slots = torch.randperm(n, generator=g)[:Bn].contiguous() if pool else None
    st = Guarded((n, H, dv, dk), torch.float32, fill=states)
    o = Guarded((Bn, H, dv), x["v"].dtype)
    args = [x[m][:, :, 0].contiguous().to(DEV) for m in ("q", "k", "v", "log_alpha", "beta")]
    B.ll_gdr_decode_step(*args, st.view, scale=0.25, slots=None if slots is None else slots.to(DEV), o=o.view)
    assert B.ll_last_device_error() == 0 and st.intact() and o.intact()
    got_o, got_s = o.view.float().cpu().numpy(), st.view.cpu().numpy()
    used = slots.tolist() if pool else list(range(Bn))
    tol = TOL_F32 if io == "f32" else 2.0 ** -8 + TOL_F32
    x["state_in"] = states[used]
    for (i, b, h, hk, lo, hi), a, _, s0, _ in slices({m: t for m, t in x.items() if m != "dstate_out"}, None):
        ro, rs = gdr.forward(*a, scale=0.25, state=s0)
        assert rel_err(got_o[b, h], ro[0], 0) <= tol
        assert rel_err(got_s[used[b], h], rs, 0) <= TOL_F32
    rest = [i for i in range(n) if i not in used]
    assert np.array_equal(got_s[rest], states.numpy()[rest])


def test_decode_padding_rows_and_bad_slots(B):
    H, d = 2, 128
    x = {n: t.to(DEV) for n, t in draw(5, H, 1, 1, d, d, "bf16", seed=20).items()}
    args = [x[m][:, :, 0].contiguous() for m in ("q", "k", "v", "log_alpha", "beta")]
    states = torch.randn(6, H, d, d, device=DEV)

    def step(slots):
        st, o = states.clone(), torch.full((5, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
        B.ll_gdr_decode_step(*args, st, slots=torch.tensor(slots, device=DEV), o=o)
        return st, o, B.ll_last_device_error()

    st, o, err = step([4, -1, 0, -1, 2])
    assert err == 0 and (o[[1, 3]] == 7.0).all() and not (o[[0, 2, 4]] == 7.0).all(dim=-1).any()
    assert torch.equal(st[[1, 3, 5]], states[[1, 3, 5]]) and not torch.equal(st[4], states[4])
    for slots, left in (([4, 6, 0, 1, 2], 1), ([4, -2, 0, 1, 2], 1), ([4, 0, 1, 1 << 40, 2], 3)):
        st, o, err = step(slots)
        assert err == 6 and (o[left] == 7.0).all()
        assert torch.equal(st[5], states[5])
    st, o, err = step([4, 3, 0, 3, 2])  # one slot twice
    assert err == 6
    assert torch.equal(st[[1, 5]], states[[1, 5]])
    st, o, err = step([-1] * 5)
    assert err == 0 and torch.equal(st, states) and (o == 7.0).all()


def test_decode_steps_in_a_graph(B):
    H, d = 4, 64
    x = {n: t.to(DEV) for n, t in draw(3, H, 2, 6, d, d, "bf16", seed=21).items()}
    names = ("q", "k", "v", "log_alpha", "beta")
    buf = [x[m][:, :, 0].contiguous() for m in names]
    slots = torch.tensor([2, 0, 1], device=DEV)
    a, b = x["state_in"].clone(), x["state_in"].clone()
    o = torch.empty_like(buf[2])
    B.ll_gdr_decode_step(*buf, a.clone(), slots=slots, o=o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.ll_gdr_decode_step(*buf, a, slots=slots, o=o)
    for t in range(6):
        for dst, m in zip(buf, names):
            dst.copy_(x[m][:, :, t])
        want = B.ll_gdr_decode_step(*buf, b, slots=slots)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(a, b)


def test_wrapper_refusals(B):
    x = {n: t.to(DEV) for n, t in draw(2, 4, 2, 20, 32, 32, "f32", seed=22).items()}
    a = [x[m] for m in ("q", "k", "v", "log_alpha", "beta")]
    with pytest.raises(ValueError):
        B.ll_gdr_fwd(a[0].transpose(1, 2), *a[1:])
    with pytest.raises(ValueError):
        B.ll_gdr_fwd(*a[:3], a[3][:, :, :10].contiguous(), a[4])
    with pytest.raises(TypeError):
        B.ll_gdr_fwd(*a[:3], a[3].double(), a[4])
    with pytest.raises(TypeError):
        B.ll_gdr_fwd(a[0].half(), a[1].half(), a[2].half(), *a[3:])
    with pytest.raises(ValueError):
        B.ll_gdr_fwd(*a, state_in=x["state_in"][:1])
    with pytest.raises(B.LLError):  # two batch rows and packed starts
        B.ll_gdr_fwd(*a, seq_starts=torch.tensor([0, 20], dtype=torch.int32, device=DEV))
    with pytest.raises(TypeError):
        B.ll_gdr_fwd(*a, seq_starts=torch.tensor([0, 20], device=DEV))
    with pytest.raises(ValueError):
        B.ll_gdr_bwd(*a, x["dout"], grads=a[:4])
    with pytest.raises(B.LLError):  # in place on an input
        B.ll_gdr_bwd(*a, x["dout"], grads=a)
    one = [t[:, :, 0].contiguous() for t in a]
    with pytest.raises(ValueError):
        B.ll_gdr_decode_step(*one, x["state_in"][:, :2].contiguous())
    with pytest.raises(TypeError):
        B.ll_gdr_decode_step(*one, x["state_in"], slots=torch.zeros(2, dtype=torch.int32, device=DEV))
    assert B.ll_last_device_error() == 0


# ------------------------------------------------------------------ in chunks or token by token
def launches(B, x, n=0):
    Bn, Hk, T, dk = x["q"].shape
    s = B.make_gdr_shape(Bn, x["v"].shape[1], Hk, T, dk, x["v"].shape[3], n, 1.0, B._io(x["q"].dtype))
    return B.ll_gdr_fwd_launches(s), B.ll_gdr_bwd_launches(s)


# many heads, where short sequences run in chunks as well; 3 and 8 value heads to a key head
@pytest.mark.parametrize("Bn,H,Hk,T,dk,dv", [
    (4, 32, 32, 70, 128, 128), (8, 24, 8, 63, 128, 128), (16, 8, 1, 128, 128, 128), (16, 16, 16, 190, 64, 128),
    (16, 8, 4, 250, 128, 64), (2, 8, 1, 300, 128, 128)])
def test_short_sequences_of_many_heads(B, Bn, H, Hk, T, dk, dv):
    x = draw(Bn, H, Hk, T, dk, dv, seed=T)
    assert launches(B, x) == (3, 4)
    check_fwd(B, x)
    check_bwd(B, x)


@pytest.mark.parametrize("starts", [[5, 6, 6, 134, 135, 300, 428, 700], [0, 0, 0, 0, 128, 128, 256, 511, 700]])
def test_packed_many_heads(B, starts):
    n = len(starts) - 1
    x = draw(1, 32, 16, 707, 128, 128, n=n, seed=n)
    for m in ("q", "k", "v", "log_alpha", "beta", "dout"):
        x[m][:, :, starts[-1]:] = float("inf")
        x[m][:, :, :starts[0]] = float("nan")
    assert launches(B, x, n) == (3, 4)
    check_fwd(B, x, starts)
    check_bwd(B, x, starts)


def test_more_sequences_than_tokens(B):
    starts = [0] * 9 + [1] * 20 + [17] * 3 + [30] * 12
    for io in ("bf16", "f32"):
        x = draw(1, 2, 1, 33, 128, 128, io, n=len(starts) - 1, seed=5)
        check_fwd(B, x, starts)
        check_bwd(B, x, starts)


@pytest.mark.parametrize("dk,dv,lo,hi", [(128, 128, 240, 260), (64, 64, 300, 330), (64, 128, 300, 330)])
def test_both_sides_of_the_choice(B, dk, dv, lo, hi):
    for T, n in ((lo, 1), (hi, 3)):
        x = draw(1, 2, 1, T, dk, dv, seed=T)
        assert launches(B, x)[0] == n
        check_fwd(B, x)
    for T, n in (((15, 2), (16, 4)) if dk * dv > 64 * 128 else ((63, 2), (128, 4))):
        x = draw(1, 2, 1, T, dk, dv, seed=T)
        assert launches(B, x)[1] == n
        check_bwd(B, x)


@pytest.mark.parametrize("T,io", [(50, "bf16"), (500, "bf16"), (100, "f32")])
@pytest.mark.parametrize("k", [-30, 20])
def test_scaling_by_powers_of_two_is_exact(B, T, io, k):
    """Values and states scaled by 2^k scale every result by it, bit for bit:
    no operand's range is used up or lost, whatever their size."""
    d, f = 128, 2.0 ** k
    x = draw(2, 4, 2, T, d, d, io, seed=23)
    y = {n: t * f if n in ("v", "state_in") else t for n, t in x.items()}
    z = {n: t * f if n in ("dout", "dstate_out") else t for n, t in x.items()}
    o, s = gpu_fwd(B, x)
    o2, s2 = gpu_fwd(B, y)
    assert np.array_equal(o2, o * f) and np.array_equal(s2, s * f)
    g, gy, gz = gpu_bwd(B, x), gpu_bwd(B, y), gpu_bwd(B, z)
    for i, (a, b, c) in enumerate(zip(g, gy, gz)):  # dq, dk, dv, dlog_alpha, dbeta, dstate_in
        assert np.array_equal(b, a if i in (2, 5) else a * f), i
        assert np.array_equal(c, a * f), i


@pytest.mark.parametrize("f", [2.0 ** -7, 1.375])
def test_keys_of_other_lengths(B, f):
    """Short ones, and long ones with beta |k|^2 still below 2, where a transition contracts."""
    x = draw(1, 4, 2, 520, 128, 128, seed=24)
    x["k"] = x["k"] * f
    check_fwd(B, x)
    check_bwd(B, x)


@pytest.mark.parametrize("T", [9, 300])
@pytest.mark.parametrize("names", [("q",), ("k",), ("v",), ("v", "state_in"), ("dout", "dstate_out"),
                                   ("q", "k", "v", "dout")])
def test_inputs_of_zeros(B, T, names):
    x = draw(1, 2, 1, T, 128, 128, seed=31)
    for n in names:
        x[n].zero_()
    check_fwd(B, x)
    check_bwd(B, x)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_state_stays_alone(B, bad):
    starts = [0, 100, 300, 700]
    x = draw(1, 8, 4, 700, 128, 128, n=3, seed=25)
    ref_o, ref_s = gpu_fwd(B, x, starts)
    ref_g = gpu_bwd(B, x, starts)
    x["state_in"][1, 3, 5, 7] = bad
    x["dstate_out"][1, 3, 100, 2] = bad
    o, s = gpu_fwd(B, x, starts)
    g = gpu_bwd(B, x, starts)
    other = [h for h in range(8) if h != 3]
    assert not np.isfinite(s[1, 3]).all()
    for got, ref in ((o, ref_o), (g[2], ref_g[2]), (g[3], ref_g[3]), (g[4], ref_g[4])):
        assert np.array_equal(got[:, other], ref[:, other])
        assert np.array_equal(got[:, 3, :100], ref[:, 3, :100]) and np.array_equal(got[:, 3, 300:], ref[:, 3, 300:])
    for got, ref in ((s, ref_s), (g[5], ref_g[5])):
        assert np.array_equal(got[:, other], ref[:, other]) and np.array_equal(got[[0, 2], 3], ref[[0, 2], 3])
    for got, ref in ((g[0], ref_g[0]), (g[1], ref_g[1])):
        assert np.array_equal(got[:, [0, 2, 3]], ref[:, [0, 2, 3]])


@pytest.mark.parametrize("T", [60, 600])
def test_two_graphs_and_an_eager_call_at_once(B, T):
    names = ("q", "k", "v", "log_alpha", "beta")
    xs = [{n: t.to(DEV) for n, t in draw(1, 4, 2, T, 128, 128, "bf16", seed=s).items()} for s in (26, 27, 28)]

    def run(x):
        a = [x[n] for n in names]
        return [B.ll_gdr_fwd(*a, state_in=x["state_in"]), *B.ll_gdr_bwd(*a, x["dout"], state_in=x["state_in"])]

    want = [run(x) for x in xs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs[:2]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run(x))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = run(xs[2])
        torch.cuda.synchronize()
        for got, ref in zip([*outs, eager], want):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert B.ll_last_device_error() == 0


@pytest.mark.parametrize("io,H,T", [("bf16", 16, (1 << 20) + 37), ("f32", 64, (1 << 18) + 5)])
def test_more_than_two_to_the_31_elements(B, io, H, T):
    """Both ends against the recurrence over 500 tokens: log_alpha = -0.5 leaves
    e^-150 of what is 300 tokens away."""
    d, near, far = 128, 200, 500
    g = torch.Generator(device=DEV).manual_seed(29)
    dt = torch.bfloat16 if io == "bf16" else torch.float32

    def r(*s):
        return torch.randn(*s, generator=g, device=DEV, dtype=dt)

    x = dict(q=r(1, 1, T, d), k=torch.nn.functional.normalize(r(1, 1, T, d), dim=-1), v=r(1, H, T, d),
             log_alpha=torch.full((1, H, T), -0.5, device=DEV),
             beta=torch.rand(1, H, T, generator=g, device=DEV), dout=r(1, H, T, d))
    a = [x[n] for n in ("q", "k", "v", "log_alpha", "beta")]
    assert x["v"].numel() > 1 << 31
    o = B.ll_gdr_fwd(*a, scale=0.5)
    dq, dk, dv, dla, db = B.ll_gdr_bwd(*a, x["dout"], scale=0.5)
    assert B.ll_last_device_error() == 0
    for first, at in ((0, slice(0, near)), (T - far, slice(far - near, far))):
        c = {n: t[:, :, first:first + far].cpu() for n, t in x.items()}
        tol = tol_out(c)
        for (i, b, h, hk, lo, hi), aa, do, _, _ in slices(c, None):
            if h not in (0, H - 1):
                continue
            ref = gdr.backward(*aa, do, scale=0.5)
            for got, want in ((o, gdr.forward(*aa, scale=0.5)[0]), (dv, ref["dv"])):
                assert rel_err(got[0, h, first:first + far][at].float().cpu().numpy(), want[at], 0) <= tol, (h, first)
            terms = np.abs((aa[2] * ref["dv"]).sum(-1)).max()
            for got, want in ((dla, ref["dlog_alpha"]), (db, ref["dbeta"])):
                den = max(np.abs(want).max(), terms)
                assert np.abs(got[0, h, first:first + far][at].cpu().numpy() - want[at]).max() <= TOL_F32 * den
        assert torch.isfinite(dq[0, 0, first:first + far]).all() and torch.isfinite(dk[0, 0, first:first + far]).all()


def test_decode_far_into_a_pool(B):
    """A pool of more than 2^31 elements."""
    H, d, n = 32, 128, 4110
    x = draw(3, H, 16, 1, d, d, "bf16", seed=30, init=False)
    states = torch.zeros(n, H, d, d, device=DEV)
    slots = [n - 1, 2, 4097]
    x["state_in"] = 0.5 * torch.randn(3, H, d, d, generator=torch.Generator().manual_seed(4))
    for b, s in enumerate(slots):
        states[s] = x["state_in"][b].to(DEV)
    args = [x[m][:, :, 0].contiguous().to(DEV) for m in ("q", "k", "v", "log_alpha", "beta")]
    o = B.ll_gdr_decode_step(*args, states, scale=0.25, slots=torch.tensor(slots, device=DEV))
    assert B.ll_last_device_error() == 0
    for (i, b, h, hk, lo, hi), a, _, s0, _ in slices(x, None):
        ro, rs = gdr.forward(*a, scale=0.25, state=s0)
        assert rel_err(o[b, h].float().cpu().numpy(), ro[0], 0) <= 2.0 ** -8 + TOL_F32
        assert rel_err(states[slots[b], h].cpu().numpy(), rs, 0) <= TOL_F32
    rest = torch.ones(n, dtype=torch.bool)
    rest[slots] = False
    assert not states[rest.to(DEV)].any()
