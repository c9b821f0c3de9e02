"""The gated delta rule with one state per head (NumPy float64; test infrastructure only).

    S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,   o_t = scale S_t q_t

(reading R7's base model, "Log-Linear Attention" study note §3-5), token by
token, and its gradient by the reverse recurrence of the same equations.  One
(sequence, head) per call; callers loop.
"""

from __future__ import annotations

import numpy as np


def _f(*xs):
    return [np.asarray(x, np.float64) for x in xs]


def forward(q, k, v, log_alpha, beta, scale=1.0, state=None):
    """q, k [T,dk]; v [T,dv]; log_alpha, beta [T]; state [dv,dk] or None (zero).
    Returns (o [T,dv], state after the last token)."""
    q, k, v, la, b = _f(q, k, v, log_alpha, beta)
    S = np.zeros((v.shape[1], k.shape[1])) if state is None else np.array(state, np.float64)
    o = np.zeros_like(v)
    for t in range(len(q)):
        a = np.exp(la[t])
        S = a * S @ (np.eye(k.shape[1]) - b[t] * np.outer(k[t], k[t])) + b[t] * np.outer(v[t], k[t])
        o[t] = scale * (S @ q[t])
    return o, S


def backward(q, k, v, log_alpha, beta, dout, scale=1.0, state=None, dstate=None):
    """Gradients of sum(o . dout) + sum(S_T . dstate).  Returns a dict with dq,
    dk, dv, dlog_alpha, dbeta, dstate_in."""
    q, k, v, la, b, do = _f(q, k, v, log_alpha, beta, dout)
    S = np.zeros((v.shape[1], k.shape[1])) if state is None else np.array(state, np.float64)
    before = []
    for t in range(len(q)):
        before.append(S)
        S = np.exp(la[t]) * S
        S = S + np.outer(b[t] * (v[t] - S @ k[t]), k[t])
    A = np.zeros_like(S) if dstate is None else np.array(dstate, np.float64)
    g = {n: np.zeros_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dlog_alpha", la), ("dbeta", b))}
    for t in reversed(range(len(q))):
        D = np.exp(la[t]) * before[t]      # the decayed state
        e = v[t] - D @ k[t]
        St = D + b[t] * np.outer(e, k[t])
        g["dq"][t] = scale * (St.T @ do[t])
        A = A + scale * np.outer(do[t], q[t])
        du = A @ k[t]
        g["dbeta"][t] = du @ e
        de = b[t] * du
        g["dv"][t] = de
        g["dk"][t] = A.T @ (b[t] * e) - D.T @ de
        dD = A - np.outer(de, k[t])
        g["dlog_alpha"][t] = np.sum(dD * D)
        A = np.exp(la[t]) * dD
    g["dstate_in"] = A
    return g
