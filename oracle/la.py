"""Linear attention with a decay per head and rotary positions (NumPy float64;
test infrastructure only).

    S_t = alpha_t S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t

(the model under the mask M^S of the "Log-Linear Attention" study note §3-5),
token by token, and its gradient by the reverse recurrence.  One (sequence, head)
per call; callers loop.  Rotations are those of complex numbers.
"""

from __future__ import annotations

import numpy as np


def _f(*xs):
    return [np.asarray(x, np.float64) for x in xs]


def forward(q, k, v, log_alpha, scale=1.0, state=None):
    """q, k [T,dk]; v [T,dv]; log_alpha [T]; state [dv,dk] or None (zero).
    Returns (o [T,dv], state after the last token)."""
    q, k, v, la = _f(q, k, v, log_alpha)
    S = np.zeros((v.shape[1], k.shape[1])) if state is None else np.array(state, np.float64)
    o = np.zeros_like(v)
    for t in range(len(q)):
        S = np.exp(la[t]) * S + np.outer(v[t], k[t])
        o[t] = scale * (S @ q[t])
    return o, S


def backward(q, k, v, log_alpha, dout, scale=1.0, state=None, dstate=None):
    """Gradients of sum(o . dout) + sum(S_T . dstate): a dict with dq, dk, dv,
    dlog_alpha, dstate_in; and "terms" [T], the 2-norm of the products that a token's
    dlog_alpha = sum(alpha_t S_{t-1} * A_t) is the sum of."""
    q, k, v, la, do = _f(q, k, v, log_alpha, dout)
    S = np.zeros((v.shape[1], k.shape[1])) if state is None else np.array(state, np.float64)
    before = []
    for t in range(len(q)):
        before.append(S)
        S = np.exp(la[t]) * S + np.outer(v[t], k[t])
    A = np.zeros_like(S) if dstate is None else np.array(dstate, np.float64)
    g = {n: np.zeros_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dlog_alpha", la), ("terms", la))}
    for t in reversed(range(len(q))):
        a = np.exp(la[t])
        g["dq"][t] = scale * ((a * before[t] + np.outer(v[t], k[t])).T @ do[t])
        A = A + scale * np.outer(do[t], q[t])
        g["dv"][t] = A @ k[t]
        g["dk"][t] = A.T @ v[t]
        g["dlog_alpha"][t] = a * np.sum(A * before[t])
        g["terms"][t] = a * np.sqrt(np.sum((A * before[t]) ** 2))
        A = a * A
    g["dstate_in"] = A
    return g


def rope(x, positions, inv_freq, interleaved=False, amp=1.0, back=False):
    """x [..., T, d], positions broadcastable to [..., T], inv_freq [rot/2] (used as given)."""
    x = np.array(x, np.float64)
    f = np.asarray(inv_freq, np.float64)
    r = 2 * len(f)
    # whole turns are taken out before the cosine, which keeps far positions exact
    turns = np.asarray(positions, np.longdouble)[..., None] * f.astype(np.longdouble) / (2 * np.longdouble(np.pi) + np.longdouble(2.4492935982947064e-16))
    w = amp * np.exp((-2j if back else 2j) * np.pi * (turns - np.rint(turns)).astype(np.float64))
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    z = (x[..., i] + 1j * x[..., j]) * w
    x[..., i], x[..., j] = z.real, z.imag
    return x
