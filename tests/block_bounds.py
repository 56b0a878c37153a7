"""Elementwise error bounds for the operators around retention, from counting
roundings.  u = 2^-24 is the relative error of one float32 rounding.

  store(t)    half a step of the storage type: 2^-8 of the value in bf16,
              2^-24 in float32.
  complement  c = 1 - a comes from e^f (the fast exponential is off by at most
              2 + 1.173 |f| units in the last place, 2u each), one addition and
              a quotient (2 units in the last place) or, for small |f|, from
              seven series steps: at most (16 + 2.4 |f|) u of c in all, and
              4 u of 1 where c is taken as 1 - e^f.
  recurrence  every step of h adds at most four roundings (two of the step, two
              of folding a span of tokens into the carry) of a value no larger
              than m_t = a m_(t-1) + |u_t|, the recurrence of the absolute
              values.
  row sums    a sum of d values in a tree of at most 64 sequential additions
              is off by at most 64 u of the sum of absolute values.
"""
from __future__ import annotations

import numpy as np

import oracle

U = 2.0 ** -24


def store(dtype: str) -> float:
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24


def _complement_error(f, c, form):
    rel = (16 + 2.4 * np.minimum(np.abs(np.where(np.isfinite(f), f, 0.0)), 100.0)) * U
    return rel * np.abs(c) + (4 * U if form == "log" else 0.0) * (np.abs(f) >= 0.25)


def scan_bounds(x, f, form, dtype, gate=None, state_in=None):
    """(bound of y, bound of h, h, |.| recurrence m)."""
    a, c = oracle.scan_gates(f, form)
    a = np.abs(a)
    y, h = oracle.scan(x, f, form, gate, state_in)
    e_c = _complement_error(f, c, form)
    e, m = np.zeros_like(h), np.zeros_like(h)
    e_t = np.zeros(h.shape[::2])
    m_t = e_t if state_in is None else np.abs(state_in)
    for t in range(h.shape[1]):
        drive = np.abs(c[:, t] * x[:, t]) if form == "logit" else np.abs(x[:, t])
        e_t = a[:, t] * e_t + e_c[:, t] * (m_t + (np.abs(x[:, t]) if form == "logit" else 0.0))
        m_t = a[:, t] * m_t + drive
        e_t = e_t + 4 * U * m_t
        e[:, t], m[:, t] = e_t, m_t
    scale = 1.0 if gate is None else np.abs(y) / np.maximum(np.abs(h), 1e-300)
    # the swish: exponential, addition, quotient and two products
    e_y = e * scale + (0 if gate is None else (24 + 2.4 * np.abs(gate)) * U * np.abs(y))
    return store(dtype) * np.abs(y) + 1.01 * e_y + 1e-37, e + 1e-37, h, m


def scan_backward_bounds(x, f, form, dtype, d_y, gate=None, state_in=None, d_state_out=None):
    """Bounds of (dx, df, dgate, d_state_in)."""
    a, c = oracle.scan_gates(f, form)
    e_c = _complement_error(f, c, form)
    _, e_h, h, _ = scan_bounds(x, f, form, "f32", None, state_in)
    before = oracle.entering(h, state_in)
    e_before = oracle.entering(e_h)
    dx, df, dg, ds = oracle.scan_backward(x, f, form, d_y, gate, state_in, d_state_out)
    sw = 1.0 if gate is None else gate / (1 + np.exp(-gate))
    slope_err = np.zeros_like(h) if gate is None else (24 + 2.4 * np.abs(gate)) * U
    d_h = np.abs(d_y * sw)
    flow_e = np.zeros(h.shape[::2])
    flow_m = flow_e if d_state_out is None else np.abs(d_state_out)
    b_x, b_f = np.zeros_like(h), np.zeros_like(h)
    aa = np.abs(a)
    for t in range(h.shape[1] - 1, -1, -1):
        e_g = flow_e + slope_err[:, t] * d_h[:, t]
        m_g = flow_m + d_h[:, t]
        e_g = e_g + 4 * U * m_g
        flow_e = aa[:, t] * e_g + e_c[:, t] * m_g + 4 * U * aa[:, t] * m_g
        # |1 - c| below one rounding of 1 is known to that rounding only
        flow_e = flow_e + U * m_g * (np.abs(c[:, t]) > 0.5)
        flow_m = aa[:, t] * m_g
        if form == "logit":
            b_x[:, t] = np.abs(c[:, t]) * e_g + e_c[:, t] * m_g + 2 * U * np.abs(c[:, t]) * m_g
            lever = np.abs(before[:, t] - x[:, t])
            b_f[:, t] = (e_before[:, t] + U * lever) * np.abs(c[:, t]) * flow_m + lever * (
                np.abs(c[:, t]) * flow_e + (e_c[:, t] + 3 * U * np.abs(c[:, t])) * flow_m)
        else:
            b_x[:, t] = e_g
            b_f[:, t] = (e_before[:, t] * flow_m
                         + np.abs(before[:, t]) * (flow_e + 3 * U * flow_m))
    s = store(dtype)
    b_g = None
    if gate is not None:
        slope = 1 / (1 + np.exp(-gate))
        slope = np.abs(slope * (1 + gate * (1 - slope)))
        b_g = s * np.abs(dg) + 1.01 * np.abs(d_y) * (
            e_h * slope + np.abs(h) * (28 + 2.4 * np.abs(gate)) * U * (1 + np.abs(gate))) + 1e-37
    return (s * np.abs(dx) + 1.01 * b_x + 1e-37, s * np.abs(df) + 1.01 * b_f + 1e-37, b_g,
            flow_e + 1e-37)


K_SUM = 64 * U


def norm_bound(v, kind, eps):
    """Bound of the normalised rows: the mean is off by K of the mean |v|, the
    spread by (K + 8 u) of itself and by what the mean's error adds."""
    z, r = oracle.norm_rows(v, kind, eps)
    level = (np.abs(v).mean(-1, keepdims=True) * r) if kind == "layer" else 0.0
    return (K_SUM + 12 * U) * (np.abs(z) + level * (1 + np.abs(z))) + 2 * U * np.abs(v) * r


def norm_backward_bound(d, e_d, z, e_z, r, kind, e_r):
    """Bound of r (d - [mean d] - z mean(d z)), given the bounds of d, z and
    the relative bound e_r of r."""
    mean = lambda t: t.mean(-1, keepdims=True)  # noqa: E731
    ad, az = np.abs(d), np.abs(z)
    s2 = mean(ad * az)
    e_s2 = K_SUM * s2 + mean(ad * e_z + e_d * az)
    total = e_d + e_z * np.abs(mean(d * z)) + az * e_s2 + 4 * U * (ad + az * s2)
    size = ad + az * s2
    if kind == "layer":
        total = total + K_SUM * mean(ad) + mean(e_d)
        size = size + mean(ad)
    return r * (total + (e_r + 4 * U) * size)


def spread_error(v, kind, eps):
    """Relative bound of 1 / spread."""
    _, r = oracle.norm_rows(v, kind, eps)
    level = (np.abs(v).mean(-1, keepdims=True) * r) if kind == "layer" else 0.0
    return K_SUM + 12 * U + K_SUM * level


def within(got, want, bound):
    """The largest |got - want| / bound, 0 / 0 = 0; nan or inf must agree."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (got.shape, want.shape)
    bound = np.broadcast_to(bound, want.shape)
    if want.size == 0:
        return 0.0
    assert np.array_equal(np.isfinite(got), np.isfinite(want))
    fine = np.isfinite(want)
    return float(np.max(np.abs(got - want)[fine] / bound[fine], initial=0.0))
