"""The gated linear recurrence at the ends of its stated range: rows of more than
2^31 bytes, spans of a few tokens at any alignment, decays close to 0, values that are not finite, and
decays above 1."""
import numpy as np
import pytest

import oracle
from block_bounds import U, store, within
from test_block_gpu import no_device_error, ret, torch  # noqa: F401 (fixtures)
from test_block_gpu import Draws, host

pytestmark = pytest.mark.gpu


# --- rows of more than 2^31 bytes ----------------------------------------------------

# D elements of one token, not 16-byte aligned: single 4-byte or 2-byte accesses
WIDE = [("bf16", (1 << 30) + 2), ("bf16", (1 << 30) + 1), ("f32", (1 << 29) + 1)]


def spots(D, n=4096):
    """Where pieces of n channels are looked at: the ends, the middle, the last
    place whose distance from the row's end passes 2^31 bytes."""
    return [0, D - n, D // 2, D - (D // 2) - n // 2]


@pytest.mark.parametrize("dt,D", WIDE)
def test_scan_of_a_very_wide_row(torch, ret, dt, D):
    """What a narrow call on the same channels gives, in both directions."""
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(D)
    x, f = (torch.randn(1, 1, D, device="cuda", dtype=dtype, generator=gen) for _ in range(2))
    assert x.numel() * x.element_size() > 1 << 31
    part = lambda t, i: t[..., i:i + 4096].contiguous()  # noqa: E731
    y, cs = ret.scan(x, f, return_chunk_states=True)
    want = [ret.scan(part(x, i), part(f, i)) for i in spots(D)]
    for i, w in zip(spots(D), want):
        assert torch.equal(part(y, i), w)
    d_y, grads = y, ret.scan_backward(x, f, cs, y)
    for i, w in zip(spots(D), want):
        got = ret.scan_backward(part(x, i), part(f, i), part(cs, i), part(d_y, i))
        assert all(torch.equal(part(g, i), v) for g, v in zip(grads, got) if v is not None)


# --- spans of a few tokens of a longer sequence -----------------------------------------

@pytest.mark.parametrize("n", [1, 2, 33])
@pytest.mark.parametrize("B", [1, 3])
@pytest.mark.parametrize("dt,D,room", [("bf16", 64, 67), ("bf16", 64, 66), ("bf16", 33, 40),
                                       ("bf16", 130, 135), ("f32", 64, 67), ("f32", 31, 32)])
def test_scan_of_a_short_span(torch, ret, dt, D, room, B, n):
    """Rows of `room` elements, odd ones among them, from every start: what dense
    copies give within the bounds of both."""
    d = Draws(torch, dt, 35)
    N = 40
    flat = [d.put(d.rng.standard_normal(B * N * room + 8)) for _ in range(4)]
    for first in (0, 1, 2):
        x, f, g, d_y = (t[first:first + B * N * room].view(B, N, room)[..., :D] for t in flat)
        for at in (0, 1, N - n):
            xs, fs, gs, ds = (t[:, at:at + n] for t in (x, f, g, d_y))
            out = torch.full((B, n + 2, room), 7.0, device="cuda", dtype=x.dtype)
            y, cs = ret.scan(xs, fs, gate=gs, out=out[:, 1:n + 1, :D], return_chunk_states=True)
            h, e, _ = forward_bound(host(xs), host(fs), "logit", None)
            gh = host(gs)
            sw = gh / (1 + np.exp(-gh))
            b = np.abs(sw) * e + ((24 + 2.4 * np.abs(gh)) * U + store(dt)) * np.abs(h * sw)
            assert within(host(y), h * sw, 1.01 * b + 1e-37) <= 1
            assert (out[:, 0] == 7).all() and (out[:, n + 1] == 7).all()
            assert (out[:, :, D:] == 7).all()
            got = ret.scan_backward(xs, fs, cs, ds)
            want = oracle.scan_backward(host(xs), host(fs), "logit", host(ds))
            zero = np.zeros((B, D))
            b_x, b_f, b_s = backward_bound(host(xs), host(fs), "logit", host(ds), None, zero)
            assert within(host(got[0]), want[0], b_x + store(dt) * np.abs(want[0]) + 1e-37) <= 1
            assert within(host(got[1]), want[1], b_f + store(dt) * np.abs(want[1]) + 1e-37) <= 1
            assert within(host(got[3]), want[3], b_s + 1e-37) <= 1


# --- decays close to 0 ---------------------------------------------------------------
#
# Bounds relative to the sums of absolute values; u = 2^-24 is one float32 rounding.
#   a decay a    (10 + 2.4 |f|) u of itself: the exponential as in block_bounds, an
#                addition, a quotient (2 units of 2u), a product, and two roundings
#                in a product of decays; LOG, where a span's decay is that of the sum
#                of its f in four parts of at most eight: 9 |f| u more
#   1 - a        (12 + 2.4 |f|) u of itself
#   a step of h  three roundings (the input, a z + input in two), and for each span
#                of at least 16 tokens the two of a fold and three of a product of
#                two spans: at most 4 u of m_t = a m_(t-1) + |u_t| a step; the flow
#                out of a span, a sum of 16 products, 16 u of itself at most, of which
#                its 16 steps have 4 u each
# and 2^-125 of the largest value, below which a product of decays is no normal number.

def size(f):
    return np.where(np.isfinite(f), np.abs(f), 0.0)       # a decay of 0 is exact


def decay_error(f, form):
    return (10 + (2.4 if form == "logit" else 11.4) * size(f)) * U


def forward_bound(x, f, form, state_in):
    """(h, bound of h, m)."""
    a, c = oracle.scan_gates(f, form)
    _, h = oracle.scan(x, f, form, None, state_in)
    r = decay_error(f, form)
    u = np.abs(c * x) if form == "logit" else np.abs(x)
    e_u = u * ((12 + 2.4 * size(f)) * U if form == "logit" else 0.0)
    e, m = np.zeros_like(h), np.zeros_like(h)
    m_t = np.zeros(h.shape[::2]) if state_in is None else np.abs(state_in)
    top, e_t = 1.0 + m_t, np.zeros_like(m_t)
    for t in range(h.shape[1]):
        e_t = a[:, t] * e_t + r[:, t] * a[:, t] * m_t + e_u[:, t]
        m_t = a[:, t] * m_t + u[:, t]
        top = np.maximum(top, m_t)
        e_t = e_t + 4 * U * m_t
        e[:, t], m[:, t] = e_t + 2.0 ** -125 * top, m_t
    return h, e, m


def backward_bound(x, f, form, d_y, state_in, d_state_out):
    """Bounds of (dx, df, d_state_in), before their rounding to the storage type."""
    a, c = oracle.scan_gates(f, form)
    h, e_h, _ = forward_bound(x, f, form, state_in)
    before, e_before = oracle.entering(h, state_in), oracle.entering(e_h)
    r, r_c = decay_error(f, form), (12 + 2.4 * size(f)) * U
    m_t = np.abs(d_state_out)
    e_t, top = np.zeros_like(m_t), 1.0 + m_t
    b_x, b_f = np.zeros_like(h), np.zeros_like(h)
    for t in range(h.shape[1] - 1, -1, -1):
        m_g = m_t + np.abs(d_y[:, t])
        e_g = e_t + U * m_g
        top = np.maximum(top, m_g)
        m_t = a[:, t] * m_g
        e_t = a[:, t] * e_g + (r[:, t] + 4 * U) * m_t
        e_g, e_f = e_g + 2.0 ** -125 * top, e_t + 2.0 ** -125 * top
        if form == "logit":
            lever = np.abs(before[:, t] - x[:, t])
            e_lever = e_before[:, t] + U * lever
            b_x[:, t] = c[:, t] * (e_g + (r_c[:, t] + U) * m_g)
            b_f[:, t] = c[:, t] * (e_lever * m_t + lever * (e_f + (r_c[:, t] + 2 * U) * m_t))
        else:
            b_x[:, t] = e_g
            b_f[:, t] = e_before[:, t] * m_t + np.abs(before[:, t]) * (e_f + U * m_t)
    return b_x, b_f, e_f


def strong(d, kind, B, N, D):
    """f: strongly forgetting gates, a mixture of them with long memories, or a
    steady decay of 0.9 (whose products are small though no decay is)."""
    f = -d.rng.uniform(8.0, 20.0, (B, N, D))
    if kind == "mixed":
        keep = d.rng.random((B, N, D)) < 0.7
        f = np.where(keep, d.rng.uniform(-3.0, 9.0, (B, N, D)), f)
    return f


STRONG = [("f32", 1, 1, 33), ("f32", 2, 40, 64), ("f32", 1, 300, 31), ("bf16", 2, 300, 72),
          ("f32", 1, 700, 32), ("bf16", 1, 3000, 64), ("f32", 1, 3000, 33)]


def strong_inputs(torch, c, form, kind, seed):
    dt, B, N, D = c
    d = Draws(torch, dt, seed)
    if kind == "steady":
        f = np.full((B, N, D), np.log(9.0) if form == "logit" else np.log(0.9))
        x = np.where(np.arange(N) % 600 < 3, 1.0, 0.0)[None, :, None] * np.ones((B, N, D))
    else:
        f = strong(d, kind, B, N, D)
        if form == "log":
            f = -np.logaddexp(0.0, -f)
        x = 1e-3 * d.rng.random((B, N, D))
        x[:, ::50] = 1e3                       # large states before small inputs
    return d, d.put(x), d.put(f), d.put(1e3 * d.rng.random((B, D)), torch.float32)


@pytest.mark.parametrize("kind", ["strong", "mixed", "steady"])
@pytest.mark.parametrize("form", ["logit", "log"])
@pytest.mark.parametrize("c", STRONG, ids=lambda c: "-".join(map(str, c)))
def test_scan_with_decays_close_to_0(torch, ret, c, form, kind):
    """Every input is positive, so the bounds are relative to each value itself."""
    d, x, f, s0 = strong_inputs(torch, c, form, kind, 31)
    y, s, cs = ret.scan(x, f, form=form, state_in=s0, return_state=True, return_chunk_states=True)
    h, e, m = forward_bound(host(x), host(f), form, host(s0))
    assert (m == h).all()
    assert within(host(y), h, e + store(c[0]) * np.abs(h)) <= 1
    assert within(host(s), h[:, -1], e[:, -1]) <= 1
    B, N, D = c[1:]
    d_y, d_s = d.put(d.rng.random((B, N, D)) + 0.1), d.put(d.rng.random((B, D)), torch.float32)
    got = ret.scan_backward(x, f, cs, d_y, form=form, d_state_out=d_s)
    want = oracle.scan_backward(host(x), host(f), form, host(d_y), None, host(s0), host(d_s))
    b_x, b_f, b_s = backward_bound(host(x), host(f), form, host(d_y), host(s0), host(d_s))
    assert within(host(got[0]), want[0], b_x + store(c[0]) * np.abs(want[0])) <= 1
    assert within(host(got[1]), want[1], b_f + store(c[0]) * np.abs(want[1])) <= 1
    assert within(host(got[3]), want[3], b_s) <= 1


@pytest.mark.parametrize("dt,B,D", [("f32", 3, 64), ("f32", 2, 33), ("bf16", 5, 1000)])
@pytest.mark.parametrize("form", ["logit", "log"])
def test_step_with_decays_close_to_0(torch, ret, form, dt, B, D):
    d, x, f, s0 = strong_inputs(torch, (dt, B, 2, D), form, "strong", 32)
    x, f = x[:, 1], f[:, 1]
    s = s0.clone()
    y = ret.scan_step(x, f, s, form=form)
    h, e, _ = forward_bound(host(x)[:, None], host(f)[:, None], form, host(s0))
    assert within(host(s), h[:, 0], e[:, 0]) <= 1
    assert within(host(y), h[:, 0], e[:, 0] + store(dt) * np.abs(h[:, 0])) <= 1


# --- values that are not finite --------------------------------------------------------

@pytest.mark.parametrize("N", [200, 3000])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("form", ["logit", "log"])
def test_scan_of_documents_with_a_value_that_is_not_finite(torch, ret, form, value, N):
    """Two documents in a row, such an input (or gradient) in the first (the last):
    a decay of 0 drops every finite state exactly, and that value stays in its own
    channel and batch row, on its own side of where it is."""
    B, D, at, reset = 2, 40, 20, 90
    d = Draws(torch, "f32", 33)
    x, f = d.normal(B, N, D), -d.normal(B, N, D).abs()
    f[:, reset] = -np.inf
    x[:, :reset] *= 1e30                         # far larger states before the reset
    clean = ret.scan(x, f, form=form)
    alone = ret.scan(x[:, reset:], f[:, reset:], form=form)
    h, e, m = forward_bound(host(x[:, reset:]), host(f[:, reset:]), form, None)
    for y in (clean[:, reset:], alone):          # nothing of the first document is left
        assert within(host(y), h, e) <= 1
    x[1, at, 3] = value
    y = ret.scan(x, f, form=form)
    rest = torch.ones_like(y, dtype=torch.bool)
    rest[1, at:, 3] = False
    assert torch.equal(y[rest], clean[rest])
    assert not torch.isfinite(y[~rest]).any()
    x[1, at, 3] = 0.0
    _, cs = ret.scan(x, f, form=form, return_chunk_states=True)
    d_y = d.normal(B, N, D)
    clean = ret.scan_backward(x, f, cs, d_y, form=form)
    d_y[0, N - 10, 5] = value
    got = ret.scan_backward(x, f, cs, d_y, form=form)
    rest = torch.ones_like(x, dtype=torch.bool)
    rest[0, :N - 9, 5] = False
    assert torch.equal(got[0][rest], clean[0][rest])
    assert torch.equal(got[1][rest], clean[1][rest])
    assert not torch.isfinite(got[0][~rest]).any()
    assert not torch.isfinite(got[3][0, 5])


@pytest.mark.parametrize("dt,N,D", [("f32", 300, 40), ("f32", 3000, 33), ("bf16", 300, 72),
                                    ("bf16", 3000, 66), ("bf16", 700, 65)])
@pytest.mark.parametrize("gate", [False, True])
def test_scan_takes_nothing_where_the_gate_is_open(torch, ret, dt, N, D, gate):
    """f = inf in the logit form: the state stays as it is whatever x is, and neither
    x nor f has a gradient; the decay is exactly 1 for what comes after."""
    B = 2
    d = Draws(torch, dt, 36)
    x, f, g = d.normal(B, N, D), d.normal(B, N, D), d.normal(B, N, D) if gate else None
    f[:, 50:] = np.inf
    x[:, 50:] = 1e38
    # (not bit by bit: the end of a span is rounded otherwise than its tokens' states)
    y, s = ret.scan(x, f, gate=g, return_state=True)
    h, e, _ = forward_bound(host(x), host(f), "logit", None)
    gh = host(g) if gate else np.zeros((B, N, D))
    sw = gh / (1 + np.exp(-gh)) if gate else 1.0
    b = np.abs(sw) * e + ((24 + 2.4 * np.abs(gh)) * U + store(dt)) * np.abs(h * sw)
    assert within(host(y), h * sw, 1.01 * b + 1e-37) <= 1
    assert within(host(s), h[:, -1], e[:, -1]) <= 1
    _, cs = ret.scan(x, f, return_chunk_states=True)
    d_y = d.normal(B, N, D)
    got = ret.scan_backward(x, f, cs, d_y, gate=g)
    assert not got[0][:, 50:].any() and not got[1][:, 50:].any()
    step = s.clone()
    ret.scan_step(x[:, 60], f[:, 60], step)
    assert torch.equal(step, s)


# --- growth ---------------------------------------------------------------------------

@pytest.mark.parametrize("dt,N,D", [("f32", 700, 40), ("bf16", 3000, 72), ("f32", 3000, 33)])
@pytest.mark.parametrize("grow", [0.5, 6.0])
def test_scan_of_growing_decays_over_a_zero_state(torch, ret, dt, N, D, grow):
    """f > 0 whose products over a span, or over a few tokens, no float32 holds: a
    zero state stays zero there, a decay of 0 ends the growth, and so do the
    gradients behind a last such token."""
    B, quiet = 2, N - 200
    d = Draws(torch, dt, 34)
    x, f = d.normal(B, N, D), -d.normal(B, N, D).abs()
    x[:, :quiet], f[:, :quiet] = 0.0, grow
    y, s, cs = ret.scan(x, f, form="log", return_state=True, return_chunk_states=True)
    h, e, _ = forward_bound(host(x[:, quiet:]), host(f[:, quiet:]), "log", None)
    assert not y[:, :quiet].any() and not cs[:, :quiet // ret.SCAN_CHUNK].any()
    assert within(host(y[:, quiet:]), h, e + store(dt) * np.abs(h) + 1e-37) <= 1
    assert within(host(s), h[:, -1], e[:, -1]) <= 1
    # growth between two decays of 0, in both directions
    x, f, d_y = d.normal(B, N, D), -d.normal(B, N, D).abs(), d.normal(B, N, D)
    quiet = np.zeros(N, bool)
    for i, k in ((20, 60), (300, 560)):
        quiet[i:k] = True
        x[:, i:k], f[:, i:k], d_y[:, i:k] = 0.0, grow, 0.0
        f[:, i], f[:, k] = -np.inf, -np.inf
    y, cs = ret.scan(x, f, form="log", return_chunk_states=True)
    h, e, _ = forward_bound(host(x), host(f), "log", None)
    assert within(host(y), h, e + store(dt) * np.abs(h) + 1e-37) <= 1
    assert not host(y)[:, quiet].any()
    zero = np.zeros((B, D))
    got = ret.scan_backward(x, f, cs, d_y, form="log")
    want = oracle.scan_backward(host(x), host(f), "log", host(d_y))
    b_x, b_f, b_s = backward_bound(host(x), host(f), "log", host(d_y), None, zero)
    assert within(host(got[0]), want[0], b_x + store(dt) * np.abs(want[0]) + 1e-37) <= 1
    assert within(host(got[1]), want[1], b_f + store(dt) * np.abs(want[1]) + 1e-37) <= 1
    assert within(host(got[3]), want[3], b_s + 1e-37) <= 1
    assert not host(got[0])[:, quiet].any()
