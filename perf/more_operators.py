"""Cases of linear attention with a decay for each head, and of the rotary
positions of its queries and keys, for timing and comparison.

    S_t = alpha_t S_{t-1} + v_t k_t^T      S_t [dv, dk]
    o_t = scale S_t q_t

fwd   the chunk-wise forward over whole sequences (``ll_la_fwd``): prompts and
      training batches, padded to one length or packed with their starts, from
      and to recurrent states; log alpha for every token, or one for a head
bwd   its gradient (``ll_la_bwd``): dq, dk, dv, d log alpha and, with a state on
      entry, that state's gradient
step  one token for every row of a batch (``ll_la_decode_step``), the states in
      a pool that a slot per row points into, queries and keys turned on the way
rope  rotary positions of queries and keys (``ll_rope_fwd``) and of their
      gradients (``ll_rope_bwd``)

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
        # a short prompt of one request, 32 value heads on 16 key heads, its state kept: a latency case
        dict(name="fwd_prompt_t77", op="fwd", io="bf16", B=1, H=32, Hk=16, T=77, dk=128, dv=128, per_head=True, seqs=0, init=False, final=True),
        # the d = 64 training shape of the forward's configurations
        dict(name="fwd_train_b2_t2048_d64", op="fwd", io="bf16", B=2, H=8, Hk=8, T=2048, dk=64, dv=64, per_head=False, seqs=0, init=False, final=False),
        # the training batch of the d = 128 configurations
        dict(name="fwd_train_b2_t4096", op="fwd", io="bf16", B=2, H=16, Hk=16, T=4096, dk=128, dv=128, per_head=False, seqs=0, init=False, final=False),
        # a long document in one pass, constant decays, its state kept for decoding
        dict(name="fwd_long_t16384", op="fwd", io="bf16", B=1, H=16, Hk=16, T=16384, dk=128, dv=128, per_head=True, seqs=0, init=False, final=True),
        # ragged requests of a serving batch, packed, resumed from their states
        dict(name="fwd_packed_13_t8191", op="fwd", io="bf16", B=1, H=16, Hk=8, T=8191, dk=128, dv=128, per_head=False, seqs=13, init=True, final=True),
        # the training step's gradient
        dict(name="bwd_train_b2_t4096", op="bwd", io="bf16", B=2, H=16, Hk=16, T=4096, dk=128, dv=128, per_head=False, seqs=0, init=False, final=False),
        # packed documents, shared key heads, constant decays, states in and their gradients out
        dict(name="bwd_packed_7_t5003", op="bwd", io="bf16", B=1, H=16, Hk=8, T=5003, dk=128, dv=128, per_head=True, seqs=7, init=True, final=True),
        # float32 io of an odd length, unequal head sizes
        dict(name="bwd_f32_t1001", op="bwd", io="f32", B=2, H=4, Hk=2, T=1001, dk=32, dv=64, per_head=False, seqs=0, init=True, final=True),
        # one token of one request
        dict(name="step_b1", op="step", io="bf16", B=1, H=32, Hk=16, T=1, dk=128, dv=128, per_head=True, pool=4, rot=128, inter=False),
        # one token of the decode configuration's batch, in rows of a larger pool
        dict(name="step_b64_pool96", op="step", io="bf16", B=64, H=32, Hk=32, T=1, dk=128, dv=128, per_head=True, pool=96, rot=64, inter=False),
        # queries and keys of the training batch
        dict(name="rope_train_b2_t4096", op="rope", io="bf16", B=2, H=16, Hk=16, T=4096, dk=128, rot=128, inter=False, scaled=False, far=0, back=False),
        # gradients of a long document far into a scaled context, a part of the head, interleaved pairs, an odd length
        dict(name="rope_back_far_t8191", op="rope", io="bf16", B=1, H=16, Hk=8, T=8191, dk=128, rot=96, inter=True, scaled=True, far=1000003, back=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "rope"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    Hk = rng.choice([1, 2, 4, 8, 16])
    H = Hk * rng.choice([1, 1, 2, 4])
    dk, dv = rng.choice([(128, 128), (128, 128), (128, 128), (64, 64), (64, 128), (32, 16)])
    c = dict(op=op, io=io, H=H, Hk=Hk, dk=dk)
    if op in ("step", "rope"):
        c.update(rot=2 * rng.randrange(1, dk // 2 + 1) if rng.random() < 0.4 else dk, inter=rng.random() < 0.5)
    if op == "rope":
        c.update(scaled=rng.random() < 0.5, far=_log(rng, 1, 4000000) if rng.random() < 0.5 else 0, back=rng.random() < 0.5)
        c["T"] = 1 if rng.random() < 0.2 else _log(rng, 1, min(16384, 131072 // H))
        return dict(c, B=_log(rng, 1, max(1, min(64, 131072 // (H * c["T"])))))
    c.update(dv=dv, per_head=rng.random() < 0.5)
    if op == "step":
        c["B"] = _log(rng, 1, max(1, min(200, 64 * 32 // H)))
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
    products (the update and S q: 4 dk dv a token and head; its gradient, both
    recurrences and three more products: 10).  A rotation: 3 a rotated element."""
    c = case
    es = 2 if c["io"] == "bf16" else 4
    rows, krows = c["B"] * c["H"] * c["T"], c["B"] * c["Hk"] * c["T"]
    if c["op"] == "rope":
        n = rows + krows
        return {"bytes": 2 * n * c["dk"] * es + 8 * c["B"] * c["T"], "flops": 3 * n * c["rot"]}
    st = 4 * c["H"] * c["dk"] * c["dv"]
    qk, vo = 2 * krows * c["dk"] * es, rows * c["dv"] * es
    gates = 4 * c["H"] if c["per_head"] else 4 * rows
    mac = rows * c["dk"] * c["dv"]
    if c["op"] == "step":
        return {"bytes": qk + 2 * vo + gates + 2 * c["B"] * st, "flops": 4 * mac}
    st *= c["seqs"] or c["B"]
    if c["op"] == "fwd":
        return {"bytes": qk + 2 * vo + gates + (c["init"] + c["final"]) * st, "flops": 4 * mac}
    return {"bytes": 2 * (qk + gates) + 3 * vo + (2 * c["init"] + c["final"]) * st, "flops": 10 * mac}


# ------------------------------------------------------------------ inputs
def _lengths(total, n, rng):
    """n lengths that add up to total: ragged, one of them a single token and
    (from four sequences on) one of them empty."""
    w = [rng.lognormvariate(0.0, 1.0) for _ in range(n)]
    fixed = {rng.randrange(n): 1}
    if n >= 4:
        fixed[rng.choice([i for i in range(n) if i not in fixed])] = 0
    free = [i for i in range(n) if i not in fixed]
    left = total - sum(fixed.values())
    whole = sum(w[i] for i in free)
    got = [fixed.get(i, int(w[i] * left / whole)) for i in range(n)]
    got[free[0]] += total - sum(got)
    return got


def _frequencies(rot, scaled):
    """Rotations per token, in radians: theta_i = 10000^(-2i/rot).  Scaled for a context 16 times
    as long: those that turn less than once within 4096 tokens slowed down by that factor, those
    that turn more than 32 times kept, a ramp between them."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaled:
        keep = ((4096 * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f = f * keep + f / 16 * (1 - keep)
    return f.float()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    io = torch.bfloat16 if c["io"] == "bf16" else torch.float32
    B, H, Hk, T, dk = (c[n] for n in ("B", "H", "Hk", "T", "dk"))
    step = c["op"] == "step"

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE)

    s = {"case": dict(c)}
    if c["op"] in ("step", "rope"):
        s["inv_freq"] = _frequencies(c["rot"], c.get("scaled", False)).to(DEVICE)
    if c["op"] == "rope":
        s["q"], s["k"] = normal(B, H, T, dk).to(io), normal(B, Hk, T, dk).to(io)
        s["amp"] = 0.1 * math.log(16.0) + 1.0 if c["scaled"] else 1.0
        s["positions"] = (c["far"] + torch.arange(T)[None] + 17 * torch.arange(B)[:, None]).to(DEVICE)
        return s
    dv = c["dv"]
    at = (B, Hk) if step else (B, Hk, T)
    av = (B, H) if step else (B, H, T)

    def feature(x):  # what a layer hands over: SiLU of a projection
        return (x * torch.sigmoid(x)).to(io)

    s["scale"] = dk ** -0.5
    s["q"], s["k"] = feature(normal(*at, dk)), feature(normal(*at, dk))
    s["v"] = normal(*av, dv).to(io)
    turn = torch.randperm(H, generator=g, device=DEVICE)
    if c["per_head"]:  # one half-life to a head: 1 - alpha from 2^-5 to 2^-12
        s["log_alpha"] = torch.log1p(-torch.exp2(-torch.linspace(5.0, 12.0, H, device=DEVICE)))[turn].contiguous()
    else:  # each head has its own time scale, from about one token to several hundred
        rate = torch.exp(torch.linspace(math.log(0.002), math.log(0.7), H, device=DEVICE))
        s["log_alpha"] = -rate[turn].view(1, H, *([1] * (len(av) - 2))) * torch.nn.functional.softplus(normal(*av))
    if step:
        s["states"] = normal(c["pool"], H, dv, dk)
        s["slots"] = torch.randperm(c["pool"], generator=g, device=DEVICE)[:B].contiguous()
        s["positions"] = torch.randint(0, 65536, (B,), generator=g, device=DEVICE)
        return s
    n = c["seqs"]
    s["lengths"] = _lengths(T, n, random.Random(seed)) if n else [T] * B
    if n:
        s["seq_starts"] = torch.tensor([0] + s["lengths"]).cumsum(0).to(torch.int32).to(DEVICE)
    rows = n or B
    if c["init"]:
        s["state_in"] = normal(rows, H, dv, dk)
    if c["op"] == "bwd":
        s["dout"] = normal(B, H, T, dv).to(io)
        if c["final"]:
            s["dstate_out"] = normal(rows, H, dv, dk)
    return s


def run(s):
    if own:
        return _run_own(s)
    return {"step": _plain_step, "rope": _plain_rope, "fwd": _plain_fwd, "bwd": _plain_bwd}[s["case"]["op"]](s)


def _run_own(s):
    from log_linear_attention_chunked_gb300 import binding

    c = s["case"]
    if c["op"] == "rope":
        f = binding.ll_rope_bwd if c["back"] else binding.ll_rope_fwd
        q, k = f(s["q"], s["k"], s["inv_freq"], positions=s["positions"], interleaved=c["inter"], amp=s["amp"])
        return {"q": q, "k": k}
    if c["op"] == "step":
        o = binding.ll_la_decode_step(s["q"], s["k"], s["v"], s["log_alpha"], s["states"], scale=s["scale"], slots=s["slots"],
                                      inv_freq=s["inv_freq"], positions=s["positions"], interleaved=c["inter"])
        return {"o": o, "states": s["states"]}
    more = dict(scale=s["scale"], state_in=s.get("state_in"), seq_starts=s.get("seq_starts"))
    shape = (len(s["lengths"]), c["H"], c["dv"], c["dk"])
    if c["op"] == "fwd":
        state = torch.empty(shape, device=DEVICE) if c["final"] else None
        o = binding.ll_la_fwd(s["q"], s["k"], s["v"], s["log_alpha"], state_out=state, **more)
        return {"o": o, "state": state}
    dstate = torch.empty(shape, device=DEVICE) if c["init"] else None
    got = binding.ll_la_bwd(s["q"], s["k"], s["v"], s["log_alpha"], s["dout"], dstate_out=s.get("dstate_out"), dstate_in=dstate, **more)
    return dict(zip(("dq", "dk", "dv", "dlog_alpha"), got), dstate_in=dstate)


# ------------------------------------------------------------------ the plain form: chunks of 128 tokens, 32 bits
CHUNK = 128


def _turn(x, pos, inv_freq, inter, amp=1.0, back=False):
    """x [B, h, T, d] float32, pos [B, T]: pairs of the first elements turned by pos * inv_freq."""
    half = inv_freq.numel()
    angle = pos.double()[:, None, :, None] * inv_freq.double()  # (far positions: 32 bits leave no digits)
    co, si = (amp * angle.cos()).float(), (amp * (-1.0 if back else 1.0) * angle.sin()).float()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if inter else (x[..., :half], x[..., half:2 * half])
    u, v = a * co - b * si, a * si + b * co
    turned = torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_rope(s):
    c = s["case"]
    more = (s["positions"], s["inv_freq"], c["inter"], s["amp"], c["back"])
    return {"q": _turn(s["q"].float(), *more).to(s["q"].dtype), "k": _turn(s["k"].float(), *more).to(s["k"].dtype)}


def _plain_step(s):
    c, v = s["case"], s["v"].float()
    rep = v.shape[1] // s["q"].shape[1]
    q, k = (_turn(s[n].float()[:, :, None], s["positions"][:, None], s["inv_freq"], c["inter"])[:, :, 0].repeat_interleave(rep, 1) for n in ("q", "k"))
    decay = torch.exp(s["log_alpha"]).expand(v.shape[:2])[..., None, None]
    st = s["states"][s["slots"]] * decay + v[..., None] * k[..., None, :]
    s["states"][s["slots"]] = st
    return {"o": (s["scale"] * (st * q[..., None, :]).sum(-1)).to(s["q"].dtype), "states": s["states"]}


def _places(s):
    """Where the tokens of each sequence stand once each is padded to whole
    chunks: (batch row, token) of [sequences, chunks * 128], and which are tokens."""
    n = torch.tensor(s["lengths"], device=DEVICE)
    t = torch.arange(max(1, -(-max(s["lengths"]) // CHUNK)) * CHUNK, device=DEVICE)
    real = t[None] < n[:, None]
    packed = "seq_starts" in s
    first = s["seq_starts"][:-1].long()[:, None] if packed else torch.zeros_like(n)[:, None]
    row = torch.zeros_like(n)[:, None] if packed else torch.arange(len(s["lengths"]), device=DEVICE)[:, None]
    return row.expand(real.shape), torch.where(real, first + t[None], 0), real


def _chunked(x, place, heads):
    """[B, h, T, ...] -> float32 [sequences, heads, chunks, 128, ...], zero where no token is."""
    row, tok, real = place
    x = x.transpose(1, 2)[row, tok].float() * real.view(*real.shape, *([1] * (x.dim() - 2)))
    x = x.transpose(1, 2)
    x = x.repeat_interleave(heads // x.shape[1], 1)
    return x.reshape(x.shape[0], x.shape[1], -1, CHUNK, *x.shape[3:])


def _back(x, place, like, heads):
    """The inverse of _chunked; shared heads are summed."""
    row, tok, real = place
    x = x.reshape(x.shape[0], heads, x.shape[1] // heads, -1, *x.shape[4:]).sum(2).transpose(1, 2)
    out = torch.zeros(like.shape[0], like.shape[2], heads, *x.shape[3:], device=x.device, dtype=x.dtype)
    out[row[real], tok[real]] = x[real]
    return out.transpose(1, 2).to(like.dtype).contiguous()


def _decays(g):
    """exp(g_i - g_j) for j <= i, else 0, from running log decays in 64 bits."""
    d = g[..., :, None] - g[..., None, :]
    return torch.where(torch.ones(d.shape[-2:], dtype=torch.bool, device=DEVICE).tril(), torch.exp(d.clamp_max(0.0)), 0.0).float()


def _plain_parts(s):
    """The chunks, their decays, and the state before each of them and after the last."""
    H = s["v"].shape[1]
    place = _places(s)
    q, k, v = (_chunked(s[n], place, H) for n in ("q", "k", "v"))
    la = s["log_alpha"]
    g = _chunked(la[None, :, None].expand(s["v"].shape[:3]) if la.dim() == 1 else la, place, H).double().cumsum(-1)
    decay = _decays(g)
    into = torch.exp(g).float()[..., None]  # from the chunk's start to a token
    out = torch.exp(g[..., -1:] - g).float()[..., None]  # from a token to the chunk's end
    ends = torch.nn.functional.pad(g[..., -1].cumsum(-1), (1, 0))  # at the chunks' borders
    across = _decays(ends)  # from border to border
    first = s["state_in"] if "state_in" in s else torch.zeros(*v.shape[:2], v.shape[-1], k.shape[-1], device=DEVICE)
    adds = torch.cat([first[:, :, None], v.mT @ (out * k)], 2).flatten(-2)
    states = (across @ adds).view(*adds.shape[:3], *first.shape[-2:])
    return place, H, q, k, v, decay, into, out, across, states


def _plain_fwd(s):
    place, H, q, k, v, decay, into, out, across, states = _plain_parts(s)
    o = s["scale"] * (into * (q @ states[:, :, :-1].mT) + ((q @ k.mT) * decay) @ v)
    return {"o": _back(o, place, s["v"], H), "state": states[:, :, -1].contiguous() if s["case"]["final"] else None}


def _plain_bwd(s):
    place, H, q, k, v, decay, into, out, across, states = _plain_parts(s)
    do = _chunked(s["dout"], place, H) * s["scale"]
    last = s["dstate_out"] if "dstate_out" in s else torch.zeros_like(states[:, :, -1])
    adds = torch.cat([(into * do).mT @ q, last[:, :, None]], 2).flatten(-2)
    adjoint = (across.mT @ adds).view(*adds.shape[:3], *last.shape[-2:])  # the gradient of the state at each border
    before, after = states[:, :, :-1], adjoint[:, :, 1:]
    score, reach = (q @ k.mT) * decay, (do @ v.mT) * decay
    past, future = into * (do @ before), out * (v @ after)
    dq, dk = past + reach @ k, future + reach.mT @ q
    dv = score.mT @ do + out * (k @ after.mT)
    # d log alpha of a token: every pair of a query at it or behind it and a key (or state) before it
    pair = (score * (do @ v.mT)).double().tril(-1)
    since = lambda x: x.flip(-1).cumsum(-1).flip(-1)  # noqa: E731
    dla = since(pair.sum(-1) - pair.sum(-2)) + since((past * q).sum(-1).double())
    y = (future * k).sum(-1).double()
    dla = dla + y.cumsum(-1) - y
    dla = dla + (into[..., -1, 0].double() * (before * after).double().sum((-1, -2)))[..., None]
    Hk = s["q"].shape[1]
    if s["case"]["per_head"]:
        dla = (dla * place[2].view(dla.shape[0], 1, *dla.shape[2:])).sum((0, 2, 3)).float()
    else:
        dla = _back(dla, place, s["log_alpha"], H)
    return {"dq": _back(dq, place, s["q"], Hk), "dk": _back(dk, place, s["k"], Hk), "dv": _back(dv, place, s["v"], H),
            "dlog_alpha": dla, "dstate_in": adjoint[:, :, 0].contiguous() if "state_in" in s else None}


# ------------------------------------------------------------------ the recurrence, in 64 bits
SEGMENT = 128


def _turned_pairs(x, pos, c, inv_freq, amp, sign):
    """Each pair as a complex number, times amp exp(sign i pos theta)."""
    r = c["rot"]
    y = x.clone()
    at = (torch.arange(0, r, 2, device=DEVICE), torch.arange(1, r, 2, device=DEVICE)) if c["inter"] else (torch.arange(r // 2, device=DEVICE), torch.arange(r // 2, r, device=DEVICE))
    z = torch.complex(x[..., at[0]], x[..., at[1]])
    theta = sign * pos.double()[:, None, ..., None] * inv_freq.double()
    z = z * amp * torch.polar(torch.ones_like(theta), theta)
    y[..., at[0]], y[..., at[1]] = z.real, z.imag
    return y


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f = {n: x.double() for n, x in s.items() if torch.is_tensor(x) and x.is_floating_point()}
    if c["op"] == "rope":
        return {n: _turned_pairs(f[n], s["positions"], c, s["inv_freq"], s["amp"], -1 if c["back"] else 1) for n in ("q", "k")}
    rep, scale, v = c["H"] // c["Hk"], s["scale"], f["v"]
    alpha = f["log_alpha"].exp()
    if c["op"] == "step":
        q, k = (_turned_pairs(f[n], s["positions"], c, s["inv_freq"], 1.0, 1).repeat_interleave(rep, 1) for n in ("q", "k"))
        st = f["states"]
        now = alpha.expand(c["B"], c["H"])[..., None, None] * st[s["slots"]] + torch.einsum("bhv,bhk->bhvk", v, k)
        st[s["slots"]] = now
        return {"o": scale * torch.einsum("bhvk,bhk->bhv", now, q), "states": st}
    q, k = f["q"].repeat_interleave(rep, 1), f["k"].repeat_interleave(rep, 1)
    if c["per_head"]:
        alpha = alpha[None, :, None].expand(v.shape[:3])
    lens = s["lengths"]
    if c["seqs"]:  # each sequence becomes a row, zeros behind its end
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
    q, k, v, alpha = rows(q), rows(k), rows(v), rows(alpha, 1.0)
    n, h, T = v.shape[:3]
    st = f["state_in"] if c["init"] else v.new_zeros(n, h, c["dv"], c["dk"])

    def forward(st, t):
        return alpha[:, :, t, None, None] * st + v[:, :, t, :, None] * k[:, :, t, None, :]

    if c["op"] == "fwd":
        o = torch.empty_like(v)
        for t in range(T):
            st = forward(st, t)
            o[:, :, t] = scale * (st @ q[:, :, t, :, None])[..., 0]
        return {"o": flat(o), "state": st if c["final"] else None}

    do = rows(f["dout"])
    starts = []
    for t in range(T):
        if t % SEGMENT == 0:
            starts.append(st)
        st = forward(st, t)
    ds = f["dstate_out"] if c["final"] else torch.zeros_like(st)
    dq, dk, dv, da = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(alpha)
    for seg in reversed(range(len(starts))):
        lo, hi = seg * SEGMENT, min(T, (seg + 1) * SEGMENT)
        before, st = [], starts[seg]
        for t in range(lo, hi):
            before.append(st)
            st = forward(st, t)
        for t in reversed(range(lo, hi)):
            prev, a = before[t - lo], alpha[:, :, t, None, None]
            dq[:, :, t] = scale * (st.mT @ do[:, :, t, :, None])[..., 0]
            ds = ds + scale * do[:, :, t, :, None] * q[:, :, t, None, :]
            dv[:, :, t] = (ds @ k[:, :, t, :, None])[..., 0]
            dk[:, :, t] = (ds.mT @ v[:, :, t, :, None])[..., 0]
            da[:, :, t] = a[..., 0, 0] * (ds * prev).sum((-1, -2))  # by log alpha
            ds = a * ds
            st = prev
        before.clear()

    def shared(x):
        return flat(x.reshape(n, c["Hk"], rep, *x.shape[2:]).sum(2))

    if c["per_head"]:
        real = torch.arange(T, device=DEVICE)[None] < torch.tensor(lens, device=DEVICE)[:, None]
        da = (da * real[:, None]).sum((0, 2))
    else:
        da = flat(da)
    return {"dq": shared(dq), "dk": shared(dk), "dv": flat(dv), "dlog_alpha": da, "dstate_in": ds if c["init"] else None}
