"""Cases of the gated delta rule's operators, for timing and comparison.

    S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T      S_t [dv, dk]
    o_t = scale S_t q_t

fwd   the chunk-wise forward over whole sequences (``ll_gdr_fwd``): prompts and
      training batches, padded to one length or packed with their starts, from
      and to recurrent states
bwd   its gradient (``ll_gdr_bwd``): dq, dk, dv, d log alpha, d beta and, with a
      state on entry, that state's gradient
step  one token for every row of a batch (``ll_gdr_decode_step``), the states
      in a pool that a slot per row points into

``own`` chooses between the plain form (32 bits, elementary operations) and
this package's entry points.  ``exact`` is the recurrence itself in 64 bits.
"""

import math
import random

import torch

own = False

DEVICE = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a short prompt of one request, 32 value heads on 16 key heads: a latency case
        dict(name="fwd_prompt_t77", op="fwd", io="bf16", B=1, H=32, Hk=16, T=77, dk=128, dv=128, seqs=0, init=False, final=True),
        # the d = 64 training shape of the forward's configurations
        dict(name="fwd_train_b2_t2048_d64", op="fwd", io="bf16", B=2, H=8, Hk=8, T=2048, dk=64, dv=64, seqs=0, init=False, final=False),
        # the Gated DeltaNet configuration's batch
        dict(name="fwd_train_b2_t4096", op="fwd", io="bf16", B=2, H=16, Hk=16, T=4096, dk=128, dv=128, seqs=0, init=False, final=False),
        # a long document in one pass, its state kept for decoding
        dict(name="fwd_long_t16384", op="fwd", io="bf16", B=1, H=16, Hk=16, T=16384, dk=128, dv=128, seqs=0, init=False, final=True),
        # ragged requests of a serving batch, packed, resumed from their states
        dict(name="fwd_packed_13_t8191", op="fwd", io="bf16", B=1, H=16, Hk=8, T=8191, dk=128, dv=128, seqs=13, init=True, final=True),
        # float32 io of an odd length, unequal head sizes
        dict(name="fwd_f32_t1001", op="fwd", io="f32", B=2, H=4, Hk=2, T=1001, dk=32, dv=64, seqs=0, init=True, final=True),
        # the training step's gradient at the Gated DeltaNet configuration
        dict(name="bwd_train_b2_t4096", op="bwd", io="bf16", B=2, H=16, Hk=16, T=4096, dk=128, dv=128, seqs=0, init=False, final=False),
        # packed documents, shared key heads, states in and their gradients out
        dict(name="bwd_packed_7_t5003", op="bwd", io="bf16", B=1, H=16, Hk=8, T=5003, dk=128, dv=128, seqs=7, init=True, final=True),
        # the smallest configuration, float32
        dict(name="bwd_f32_t64_d16", op="bwd", io="f32", B=1, H=2, Hk=2, T=64, dk=16, dv=16, seqs=0, init=False, final=False),
        # one token of one request
        dict(name="step_b1", op="step", io="bf16", B=1, H=32, Hk=16, T=1, dk=128, dv=128, pool=4),
        # one token of the decode configuration's batch
        dict(name="step_b64", op="step", io="bf16", B=64, H=32, Hk=32, T=1, dk=128, dv=128, pool=64),
        # a large batch with rows of a larger pool, shared key heads
        dict(name="step_b211_pool256", op="step", io="bf16", B=211, H=32, Hk=16, T=1, dk=128, dv=128, pool=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    Hk = rng.choice([1, 2, 4, 8, 16])
    H = Hk * rng.choice([1, 1, 2, 4])
    dk, dv = rng.choice([(128, 128), (128, 128), (128, 128), (64, 64), (64, 128), (32, 16)])
    c = dict(op=op, io=io, H=H, Hk=Hk, dk=dk, dv=dv)
    if op == "step":
        c["B"] = _log(rng, 1, max(1, min(211, 211 * 32 // H)))
        return dict(c, T=1, pool=c["B"] + rng.randrange(0, 40))
    rows = 262144 if op == "fwd" and io == "bf16" else 131072 if io == "bf16" else 16384  # heads x tokens at most
    # (a single token without a state on entry has d log alpha = 0 throughout)
    c["T"] = _log(rng, 1 if op == "fwd" else 2, min(16384 if op == "fwd" else 8192, rows // H))
    packed = c["T"] >= 8 and rng.random() < 0.4
    c["seqs"] = _log(rng, 2, min(24, c["T"] // 4)) if packed else 0
    c["B"] = 1 if packed else _log(rng, 1, max(1, min(16, rows // (H * c["T"]))))
    c["init"], c["final"] = rng.random() < 0.5, rng.random() < 0.5
    return c


def work(case):
    """Each input read once and each output written once; the recurrence's own
    products (S k, the update, S q: 6 dk dv a token and head; its gradient 16)."""
    c = case
    es = 2 if c["io"] == "bf16" else 4
    rows, krows, st = c["B"] * c["H"] * c["T"], c["B"] * c["Hk"] * c["T"], 4 * c["H"] * c["dk"] * c["dv"]
    qk, vo, gates = 2 * krows * c["dk"] * es, rows * c["dv"] * es, 8 * rows
    mac = rows * c["dk"] * c["dv"]
    if c["op"] == "step":
        return {"bytes": qk + 2 * vo + gates + 2 * c["B"] * st, "flops": 6 * mac}
    st *= c["seqs"] or c["B"]
    if c["op"] == "fwd":
        return {"bytes": qk + 2 * vo + gates + (c["init"] + c["final"]) * st, "flops": 6 * mac}
    return {"bytes": 2 * (qk + gates) + 3 * vo + (2 * c["init"] + c["final"]) * st, "flops": 16 * mac}


# ------------------------------------------------------------------ inputs
def _lengths(total, n, rng):
    """n lengths that add up to total: ragged, one of them a single token and
    (from four sequences on) one of them empty."""
    w = [rng.lognormvariate(0.0, 1.0) for _ in range(n)]
    fixed = {}
    if n >= 2:
        fixed[rng.randrange(n)] = 1
    if n >= 4:
        fixed[rng.choice([i for i in range(n) if i not in fixed])] = 0
    free = [i for i in range(n) if i not in fixed]
    left = total - sum(fixed.values())
    scale = left / sum(w[i] for i in free)
    got = [fixed.get(i, int(w[i] * scale)) for i in range(n)]
    got[free[0]] += total - sum(got)
    return got


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    io = torch.bfloat16 if c["io"] == "bf16" else torch.float32
    B, H, Hk, T, dk, dv = (c[n] for n in ("B", "H", "Hk", "T", "dk", "dv"))
    step = c["op"] == "step"

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE)

    def unit(x):  # what a layer hands over: SiLU, then a row of norm 1
        x = x * torch.sigmoid(x)
        return (x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-6)).to(io)

    at = (B, Hk) if step else (B, Hk, T)
    av = (B, H) if step else (B, H, T)
    s = {"case": dict(c), "scale": dk ** -0.5}
    s["q"], s["k"] = unit(normal(*at, dk)), unit(normal(*at, dk))
    s["v"] = normal(*av, dv).to(io)
    # each head has its own time scale, from about one token to several hundred
    rate = torch.exp(torch.linspace(math.log(0.002), math.log(0.7), H, device=DEVICE))
    rate = rate[torch.randperm(H, generator=g, device=DEVICE)].view(1, H, *([1] * (len(av) - 2)))
    s["log_alpha"] = -rate * torch.nn.functional.softplus(normal(*av))
    s["beta"] = torch.sigmoid(normal(*av))
    if step:
        s["states"] = 0.1 * normal(c["pool"], H, dv, dk)
        s["slots"] = torch.randperm(c["pool"], generator=g, device=DEVICE)[:B].contiguous()
        return s
    n = c["seqs"]
    s["lengths"] = _lengths(T, n, random.Random(seed)) if n else [T] * B
    if n:
        ends = torch.tensor([0] + s["lengths"]).cumsum(0).to(torch.int32)
        s["seq_starts"] = ends.to(DEVICE)
    rows = n or B
    if c["init"]:
        s["state_in"] = 0.1 * normal(rows, H, dv, dk)
    if c["op"] == "bwd":
        s["dout"] = normal(B, H, T, dv).to(io)
        if c["final"]:
            s["dstate_out"] = normal(rows, H, dv, dk)
    return s


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    return _plain_step(s) if op == "step" else _plain_fwd(s) if op == "fwd" else _plain_bwd(s)


def _run_own(s):
    from log_linear_attention_chunked_gb300 import binding

    c = s["case"]
    if c["op"] == "step":
        o = binding.ll_gdr_decode_step(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["states"], scale=s["scale"], slots=s["slots"])
        return {"o": o, "states": s["states"]}
    more = dict(scale=s["scale"], state_in=s.get("state_in"), seq_starts=s.get("seq_starts"))
    shape = (len(s["lengths"]), c["H"], c["dv"], c["dk"])
    if c["op"] == "fwd":
        state = torch.empty(shape, device=DEVICE) if c["final"] else None
        o = binding.ll_gdr_fwd(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], state_out=state, **more)
        return {"o": o, "state": state}
    dstate = torch.empty(shape, device=DEVICE) if c["init"] else None
    got = binding.ll_gdr_bwd(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["dout"], dstate_out=s.get("dstate_out"), dstate_in=dstate, **more)
    return dict(zip(("dq", "dk", "dv", "dlog_alpha", "dbeta"), got), dstate_in=dstate)


# ------------------------------------------------------------------ the plain form: chunks of 64 tokens, 32 bits
CHUNK = 64


def _plain_step(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    rep = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    st = s["states"][s["slots"]] * torch.exp(s["log_alpha"])[..., None, None]
    u = s["beta"][..., None] * (v - (st * k[..., None, :]).sum(-1))
    st = st + u[..., None] * k[..., None, :]
    s["states"][s["slots"]] = st
    return {"o": (s["scale"] * (st * q[..., None, :]).sum(-1)).to(s["q"].dtype), "states": s["states"]}


def _places(s):
    """Where the tokens of each sequence stand once each is padded to whole
    chunks: (batch row, token) of [sequences, chunks * 64], and which are tokens."""
    n = torch.tensor(s["lengths"], device=DEVICE)
    t = torch.arange(max(1, -(-max(s["lengths"]) // CHUNK)) * CHUNK, device=DEVICE)
    real = t[None] < n[:, None]
    packed = "seq_starts" in s
    first = s["seq_starts"][:-1].long()[:, None] if packed else torch.zeros_like(n)[:, None]
    row = torch.zeros_like(n)[:, None] if packed else torch.arange(len(s["lengths"]), device=DEVICE)[:, None]
    return row.expand(real.shape), torch.where(real, first + t[None], 0), real


def _chunked(x, place, heads):
    """[B, h, T, ...] -> float32 [sequences, heads, chunks, 64, ...], zero where no token is."""
    row, tok, real = place
    x = x.transpose(1, 2)[row, tok].float() * real.view(*real.shape, *([1] * (x.dim() - 2)))
    x = x.transpose(1, 2)
    x = x.repeat_interleave(heads // x.shape[1], 1)
    return x.reshape(x.shape[0], x.shape[1], -1, CHUNK, *x.shape[3:])


def _back(x, place, like, heads):
    """The inverse of _chunked; shared heads are summed."""
    row, tok, real = place
    x = x.reshape(x.shape[0], heads, x.shape[1] // heads, -1, *x.shape[4:]).sum(2).transpose(1, 2)
    out = torch.zeros(like.shape[0], like.shape[2], heads, *x.shape[3:], device=x.device)
    out[row[real], tok[real]] = x[real].float()
    return out.transpose(1, 2).to(like.dtype).contiguous()


def _plain_parts(s):
    """What a chunk needs that does not depend on the state before it."""
    H = s["v"].shape[1]
    place = _places(s)
    q, k, v, la, b = (_chunked(s[n], place, H) for n in ("q", "k", "v", "log_alpha", "beta"))
    g = la.double().cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, device=DEVICE).tril()
    decay = torch.exp((g[..., :, None] - g[..., None, :]).clamp_max(0.0)).float() * low
    kk = (k @ k.mT) * decay * low.tril(-1)
    inv = torch.eye(CHUNK, device=DEVICE).expand(kk.shape).clone()  # (I + diag(b) kk)^-1, row by row
    bk = b[..., None] * kk
    for i in range(1, CHUNK):
        inv[..., i, :i] = -(bk[..., i, None, :i] @ inv[..., :i, :i])[..., 0, :]
    score = s["scale"] * (q @ k.mT) * decay
    into = torch.exp(g).float()[..., None]  # from the chunk's start to a token
    out = torch.exp(g[..., -1:] - g).float()[..., None]  # from a token to the chunk's end
    end = torch.exp(g[..., -1]).float()[..., None, None]
    return place, H, q, k, v, b[..., None], decay, kk, inv, score, into, out, end


def _plain_scan(s, parts):
    """The states before every chunk and after the last, and the rows u that are written."""
    place, H, q, k, v, b, decay, kk, inv, score, into, out, end = parts
    st = s["state_in"] if "state_in" in s else torch.zeros(v.shape[0], H, v.shape[-1], k.shape[-1], device=DEVICE)
    states, us = [], []
    for n in range(q.shape[2]):
        u = inv[:, :, n] @ (b[:, :, n] * (v[:, :, n] - into[:, :, n] * (k[:, :, n] @ st.mT)))
        states.append(st)
        us.append(u)
        st = end[:, :, n] * st + u.mT @ (out[:, :, n] * k[:, :, n])
    return torch.stack(states, 2), st, torch.stack(us, 2)


def _plain_fwd(s):
    parts = _plain_parts(s)
    place, H, q, k, v, b, decay, kk, inv, score, into, out, end = parts
    states, last, u = _plain_scan(s, parts)
    o = s["scale"] * into * (q @ states.mT) + score @ u
    return {"o": _back(o, place, s["v"], H), "state": last if s["case"]["final"] else None}


def _plain_bwd(s):
    parts = _plain_parts(s)
    place, H, q, k, v, b, decay, kk, inv, score, into, out, end = parts
    states, last, u = _plain_scan(s, parts)
    do = _chunked(s["dout"], place, H)
    d = s["dstate_out"] if "dstate_out" in s else torch.zeros_like(last)
    after, ws = [], []
    for n in reversed(range(q.shape[2])):
        w = inv[:, :, n].mT @ (score[:, :, n].mT @ do[:, :, n] + out[:, :, n] * (k[:, :, n] @ d.mT))
        after.append(d)
        ws.append(w)
        d = end[:, :, n] * d + (s["scale"] * into[:, :, n] * do[:, :, n]).mT @ q[:, :, n] - (into[:, :, n] * b[:, :, n] * w).mT @ k[:, :, n]
    after, w = torch.stack(after[::-1], 2), torch.stack(ws[::-1], 2)
    reach = s["scale"] * (do @ u.mT) * decay
    wu = w @ u.mT
    past = into * (w @ states)  # w^T of the state before each row
    inner = b * wu * decay * torch.ones_like(decay[0, 0, 0]).tril(-1)
    dq = s["scale"] * into * (do @ states) + reach @ k
    dk = reach.mT @ q + out * (u @ after) - inner.mT @ k - b * past - inner @ k
    dv = b * w
    dbeta = (w * v).sum(-1) - (past * k).sum(-1) - (wu * kk).sum(-1)
    o = s["scale"] * into * (q @ states.mT) + score @ u
    dg = ((do * o).sum(-1) - (v * dv).sum(-1)).double()
    ends = torch.cat([states[:, :, 1:], last[:, :, None]], 2)
    dla = dg.flip(-1).cumsum(-1).flip(-1) + (ends * after).double().sum((-1, -2))[..., None]
    Hk = s["q"].shape[1]
    return {"dq": _back(dq, place, s["q"], Hk), "dk": _back(dk, place, s["k"], Hk), "dv": _back(dv, place, s["v"], H),
            "dlog_alpha": _back(dla, place, s["log_alpha"], H), "dbeta": _back(dbeta, place, s["beta"], H),
            "dstate_in": d if "state_in" in s else None}


# ------------------------------------------------------------------ the recurrence, in 64 bits
SEGMENT = 128


def exact(case, seed):
    s = prepare(case, seed)
    f = {n: x.double() for n, x in s.items() if torch.is_tensor(x) and x.is_floating_point()}
    rep = case["H"] // case["Hk"]
    scale = s["scale"]
    q, k = f["q"].repeat_interleave(rep, 1), f["k"].repeat_interleave(rep, 1)
    v, alpha, beta = f["v"], f["log_alpha"].exp(), f["beta"]
    if case["op"] == "step":
        st = f["states"]
        now = alpha[..., None, None] * st[s["slots"]]
        e = v - torch.einsum("bhvk,bhk->bhv", now, k)
        now = now + torch.einsum("bhv,bhk->bhvk", beta[..., None] * e, k)
        st[s["slots"]] = now
        return {"o": scale * torch.einsum("bhvk,bhk->bhv", now, q), "states": st}

    lens = s["lengths"]
    if case["seqs"]:  # each sequence becomes a row, zeros behind its end
        pad, at = max(1, max(lens)), [sum(lens[:i]) for i in range(len(lens))]

        def rows(x, fill=0.0):
            y = x.new_full((len(lens), x.shape[1], pad, *x.shape[3:]), fill)
            for i, (a, n) in enumerate(zip(at, lens)):
                y[i, :, :n] = x[0, :, a:a + n]
            return y

        def flat(y):
            return torch.cat([y[i, :, :n] for i, n in enumerate(lens)], 1)[None]
    else:
        def rows(x, fill=0.0):
            return x

        def flat(y):
            return y
    q, k, v, beta, alpha = rows(q), rows(k), rows(v), rows(beta), rows(alpha, 1.0)
    n, h, T = v.shape[:3]
    st = f["state_in"] if case["init"] else v.new_zeros(n, h, case["dv"], case["dk"])

    def forward(st, t):
        a = alpha[:, :, t, None, None] * st
        e = v[:, :, t] - (a @ k[:, :, t, :, None])[..., 0]
        return a + (beta[:, :, t, None] * e)[..., None] * k[:, :, t, None, :], e

    if case["op"] == "fwd":
        o = torch.empty_like(v)
        for t in range(T):
            st, _ = forward(st, t)
            o[:, :, t] = scale * (st @ q[:, :, t, :, None])[..., 0]
        return {"o": flat(o), "state": st if case["final"] else None}

    do = rows(f["dout"])
    starts = []
    for t in range(T):
        if t % SEGMENT == 0:
            starts.append(st)
        st, _ = forward(st, t)
    ds = f["dstate_out"] if case["final"] else torch.zeros_like(st)
    dq, dk, dv, da, db = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(alpha), torch.zeros_like(beta)
    for seg in reversed(range(len(starts))):
        lo, hi = seg * SEGMENT, min(T, (seg + 1) * SEGMENT)
        before, errs, st = [], [], starts[seg]
        for t in range(lo, hi):
            before.append(st)
            st, e = forward(st, t)
            errs.append(e)
        for t in reversed(range(lo, hi)):
            prev, e, kt, bt = before[t - lo], errs[t - lo], k[:, :, t], beta[:, :, t, None]
            dq[:, :, t] = scale * (st.mT @ do[:, :, t, :, None])[..., 0]
            ds = ds + scale * do[:, :, t, :, None] * q[:, :, t, None, :]
            dsk = (ds @ kt[..., None])[..., 0]
            decayed = alpha[:, :, t, None, None] * prev
            de = bt * dsk  # the gradient of e = v - decayed k
            dv[:, :, t] = de
            db[:, :, t] = (dsk * e).sum(-1)
            dk[:, :, t] = (ds.mT @ (bt * e)[..., None])[..., 0] - (decayed.mT @ de[..., None])[..., 0]
            ddec = ds - de[..., None] * kt[:, :, None, :]
            da[:, :, t] = (ddec * decayed).sum((-1, -2))  # by log alpha
            ds = alpha[:, :, t, None, None] * ddec
            st = prev
        before.clear()

    def shared(x):
        return flat(x.reshape(n, case["Hk"], rep, *x.shape[2:]).sum(2))

    return {"dq": shared(dq), "dk": shared(dk), "dv": flat(dv), "dlog_alpha": flat(da), "dbeta": flat(db), "dstate_in": ds if case["init"] else None}
