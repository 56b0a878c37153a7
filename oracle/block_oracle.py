"""CPU oracle for the operators around retention, float64 numpy: the gated
linear recurrence, the per-head norm with its output gate, the residual sum
with the norms around it, and the backward of each.

TEST INFRASTRUCTURE ONLY, like retention_oracle.py; it shares no code with the
CUDA path.  The functions follow the definitions in include/retention.h token
by token and row by row.

  [RetNet blog]  "RetNet - Retentive Network - A Successor to Transformer for
                 LLMs" (irregular6612.github.io): Key Equations (recurrent
                 form), core components (norm and swish gating), framework
                 graph (residuals and norms of the block).
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def _swish(g):
    return g * _sigmoid(g)


def _swish_slope(g):
    s = _sigmoid(g)
    return s + g * s * (1.0 - s)


def scan_gates(f, form: str):
    """The decay a and its complement 1 - a."""
    if form == "logit":
        return _sigmoid(f), _sigmoid(-f)
    return np.exp(f), -np.expm1(f)


def scan(x, f, form: str, gate=None, state_in=None):
    """(y, h): x, f, gate [B,N,D]; state_in [B,D] or None; h [B,N,D] holds the
    state after every token."""
    x, f, gate, state_in = _f64(x), _f64(f), _f64(gate), _f64(state_in)
    a, c = scan_gates(f, form)
    h = np.zeros_like(x)
    past = np.zeros(x.shape[::2]) if state_in is None else state_in
    for t in range(x.shape[1]):
        past = a[:, t] * past + (c[:, t] * x[:, t] if form == "logit" else x[:, t])
        h[:, t] = past
    return (h if gate is None else h * _swish(gate)), h


def entering(h, state_in=None):
    """The state before every token, given the one after every token."""
    first = np.zeros_like(h[:, :1]) if state_in is None else _f64(state_in)[:, None]
    return np.concatenate([first, h[:, :-1]], axis=1)


def scan_backward(x, f, form: str, d_y, gate=None, state_in=None, d_state_out=None):
    """(dx, df, dgate or None, d_state_in)."""
    x, f, gate, d_y = _f64(x), _f64(f), _f64(gate), _f64(d_y)
    _, h = scan(x, f, form, None, state_in)
    before = entering(h, state_in)
    a, c = scan_gates(f, form)
    d_h = d_y if gate is None else d_y * _swish(gate)
    flow = np.zeros(x.shape[::2]) if d_state_out is None else _f64(d_state_out)
    dx, df = np.zeros_like(x), np.zeros_like(x)
    for t in range(x.shape[1] - 1, -1, -1):
        G = d_h[:, t] + flow
        if form == "logit":
            dx[:, t] = c[:, t] * G
            df[:, t] = G * (before[:, t] - x[:, t]) * a[:, t] * c[:, t]
        else:
            dx[:, t] = G
            df[:, t] = G * before[:, t] * a[:, t]
        flow = a[:, t] * G
    return dx, df, None if gate is None else d_y * h * _swish_slope(gate), flow


def norm_rows(v, kind: str, eps: float):
    """(normalised rows, 1 / spread): over the last axis, biased."""
    v = _f64(v)
    if kind == "layer":
        v = v - v.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return v * r, r


def norm_rows_backward(d_hat, hat, r, kind: str):
    out = d_hat - hat * (d_hat * hat).mean(-1, keepdims=True)
    if kind == "layer":
        out = out - d_hat.mean(-1, keepdims=True)
    return r * out


def norm_gate(y, gate, kind: str, eps: float, token_major: bool = False):
    z, _ = norm_rows(y, kind, eps)
    if token_major:
        z = np.swapaxes(z, 1, 2)
    return z if gate is None else z * _swish(_f64(gate))


def norm_gate_backward(y, gate, d_o, kind: str, eps: float, token_major: bool = False):
    """(dy, dgate or None)."""
    z, r = norm_rows(y, kind, eps)
    gate, d = _f64(gate), _f64(d_o)
    d_gate = None
    if gate is not None:
        d_gate = d * (np.swapaxes(z, 1, 2) if token_major else z) * _swish_slope(gate)
        d = d * _swish(gate)
    if token_major:
        d = np.swapaxes(d, 1, 2)
    return norm_rows_backward(d, z, r, kind), d_gate


def add_norm(x, residual, w, w_post, post_norm, norm: str, alpha: float, beta: float, eps: float):
    """(res_out, y)."""
    u = _f64(x)
    if post_norm is not None:
        u, _ = norm_rows(u, post_norm, eps)
    if w_post is not None:
        u = u * _f64(w_post)
    r = beta * u if residual is None else alpha * _f64(residual) + beta * u
    y, _ = norm_rows(r, norm, eps)
    return r, y if w is None else y * _f64(w)


def add_norm_backward(x, res_out, w, d_y, d_res_out, w_post, post_norm, norm: str, alpha: float,
                      beta: float, eps: float):
    """(dx, dresidual, dw, dw_post) from the stored sum res_out."""
    hat, r = norm_rows(res_out, norm, eps)
    d_y = _f64(d_y)
    rows = tuple(range(d_y.ndim - 1))
    dw = (d_y * hat).sum(rows)
    d = norm_rows_backward(d_y if w is None else d_y * _f64(w), hat, r, norm)
    if d_res_out is not None:
        d = d + _f64(d_res_out)
    du = beta * d
    if post_norm is not None:
        xh, rx = norm_rows(x, post_norm, eps)
    else:
        xh = _f64(x)
    dw_post = None if x is None else (du * xh).sum(rows)
    dx = du if w_post is None else du * _f64(w_post)
    if post_norm is not None:
        dx = norm_rows_backward(dx, xh, rx, post_norm)
    return dx, alpha * d, dw, dw_post
