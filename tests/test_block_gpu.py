"""The gated linear recurrence, the norm-and-gate pass and the residual-and-norm
pass on the GPU against the float64 oracle, element by element within the
bounds of block_bounds.py."""
import numpy as np
import pytest

import oracle
from block_bounds import (K_SUM, U, norm_backward_bound, norm_bound, scan_backward_bounds,
                          scan_bounds, spread_error, store, within)

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


@pytest.fixture(scope="module")
def ret(torch):
    import linear_recurrent_sequence_scale_b200 as ret
    ret.load_library()
    return ret


@pytest.fixture(autouse=True)
def no_device_error(ret):
    yield
    assert ret.device_error() == 0


def dtype_of(torch, dt):
    return torch.bfloat16 if dt == "bf16" else torch.float32


def host(t):
    return t.detach().double().cpu().numpy()


class Draws:
    """Seeded tensors on the device, in the storage type, with their float64 values."""

    def __init__(self, torch, dt, seed):
        self.torch, self.dt = torch, dtype_of(torch, dt)
        self.rng = np.random.default_rng(seed)

    def put(self, a, dtype=None):
        t = self.torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype or self.dt)
        return t

    def normal(self, *shape, dtype=None):
        return self.put(self.rng.standard_normal(shape), dtype)

    def f32(self, *shape):
        return self.normal(*shape, dtype=self.torch.float32)


def forget(d, form, B, N, D, resets):
    tau = np.exp(d.rng.uniform(np.log(2.0), np.log(1000.0), D))
    n = d.rng.standard_normal((B, N, D))
    f = np.log(tau) + n if form == "logit" else -np.log1p(np.exp(n)) / tau
    if form == "log" and N > 2:
        f[:, N // 2] = -30.0 * d.rng.random(D)      # strong decays too
    if resets:
        f[:, d.rng.integers(0, N, max(1, N // 60))] = -np.inf
    return d.put(f)


def scan_inputs(torch, c, seed=1):
    dt, form, B, N, D = c["dt"], c["form"], c["B"], c["N"], c["D"]
    d = Draws(torch, dt, seed)
    x, f = d.normal(B, N, D), forget(d, form, B, N, D, c.get("resets", True))
    g = 2 * d.normal(B, N, D) if c["gate"] else None
    if c.get("fused"):
        p = torch.cat([x, f] + ([g] if g is not None else []), -1)
        x, f = p[..., :D], p[..., D:2 * D]
        g = p[..., 2 * D:] if g is not None else None
    s0 = d.f32(B, D) if c["state"] else None
    return d, x, f, g, s0


def opt(t):
    return None if t is None else host(t)


def case(dt, form, B, N, D, gate=False, state=False, fused=False, **kw):
    return dict(dt=dt, form=form, B=B, N=N, D=D, gate=gate, state=state, fused=fused, **kw)


SCAN = [
    case("f32", "logit", 1, 1, 1), case("bf16", "log", 1, 1, 8, state=True),
    case("bf16", "logit", 2, 3, 64, gate=True, state=True),
    case("f32", "log", 1, 64, 32, state=True), case("f32", "logit", 1, 65, 33, gate=True),
    case("bf16", "logit", 1, 127, 128, state=True), case("bf16", "log", 3, 128, 40, gate=True),
    case("bf16", "logit", 1, 129, 72, fused=True, state=True),
    case("bf16", "logit", 2, 257, 96, gate=True, fused=True),
    case("f32", "log", 2, 300, 100, gate=True, state=True, fused=True),
    case("bf16", "log", 1, 513, 65, state=True), case("f32", "logit", 3, 511, 31),
    case("bf16", "log", 2, 1000, 257, gate=True, state=True, fused=True),
    case("bf16", "logit", 1, 2049, 512, gate=True, state=True),
    case("f32", "log", 1, 4100, 64, state=True),
    case("bf16", "log", 1, 9000, 64, gate=True, state=True),
    case("f32", "logit", 5, 700, 1001, gate=True, state=True, fused=True),
    # too long for whole pieces: items dealt over the blocks, at every alignment
    case("bf16", "logit", 2, 3001, 72, state=True, fused=True),
    case("bf16", "logit", 2, 3001, 65, gate=True), case("bf16", "log", 1, 2817, 130, state=True),
    case("f32", "logit", 1, 2819, 31, state=True), case("f32", "log", 3, 2690, 36, gate=True),
]
ids = lambda c: "-".join(str(v) for v in c.values())  # noqa: E731


@pytest.mark.parametrize("c", SCAN, ids=ids)
def test_scan(torch, ret, c):
    d, x, f, g, s0 = scan_inputs(torch, c)
    y, s, cs = ret.scan(x, f, form=c["form"], gate=g, state_in=s0, return_state=True,
                        return_chunk_states=True)
    again = ret.scan(x, f, form=c["form"], gate=g, state_in=s0)
    b_y, b_h, h, _ = scan_bounds(host(x), host(f), c["form"], c["dt"], opt(g), opt(s0))
    want, _ = oracle.scan(host(x), host(f), c["form"], opt(g), opt(s0))
    assert within(host(y), want, b_y) <= 1
    assert within(host(s), h[:, -1], b_h[:, -1]) <= 1
    before = oracle.entering(h, opt(s0))[:, ::ret.SCAN_CHUNK]
    assert within(host(cs), before, oracle.entering(b_h)[:, ::ret.SCAN_CHUNK] + 1e-37) <= 1
    assert torch.equal(y, again)          # the same bits, with and without the extra outputs


@pytest.mark.parametrize("c", SCAN, ids=ids)
def test_scan_backward(torch, ret, c):
    d, x, f, g, s0 = scan_inputs(torch, c, seed=2)
    B, N, D = c["B"], c["N"], c["D"]
    d_y, d_s = d.normal(B, N, D), d.f32(B, D) if c["state"] else None
    _, cs = ret.scan(x, f, form=c["form"], state_in=s0, return_chunk_states=True)
    out = {}
    if c["fused"]:                        # gradients side by side, for the projection's backward
        p = torch.full((B, N, (3 if c["gate"] else 2) * D), 7.0, device="cuda", dtype=x.dtype)
        out = dict(grad_x=p[..., :D], grad_f=p[..., D:2 * D])
        if c["gate"]:
            out["grad_gate"] = p[..., 2 * D:]
    got = ret.scan_backward(x, f, cs, d_y, form=c["form"], gate=g, d_state_out=d_s, **out)
    args = (host(d_y), opt(g), opt(s0), opt(d_s))
    want = oracle.scan_backward(host(x), host(f), c["form"], *args)
    bound = scan_backward_bounds(host(x), host(f), c["form"], c["dt"], *args)
    for name, a, w, b in zip(("x", "f", "gate", "state"), got, want, bound):
        if w is None:
            assert a is None
        else:
            assert within(host(a), w, b) <= 1, name
    twice = ret.scan_backward(x, f, cs, d_y, form=c["form"], gate=g, d_state_out=d_s)
    assert all(torch.equal(a, b) for a, b in zip(got, twice) if a is not None)


@pytest.mark.parametrize("c", [
    case("bf16", "logit", 1, 1, 1), case("bf16", "log", 8, 1, 4096, gate=True, fused=True),
    case("f32", "logit", 3, 1, 33, gate=True), case("bf16", "log", 17, 1, 100, fused=True),
    case("f32", "log", 300, 1, 256), case("bf16", "logit", 2, 1, 1003, gate=True, fused=True),
], ids=ids)
def test_scan_step(torch, ret, c):
    d, x, f, g, _ = scan_inputs(torch, c | dict(resets=False), seed=3)
    x, f, g = (None if t is None else t[:, 0] for t in (x, f, g))
    s0 = d.f32(c["B"], c["D"])
    put = torch.empty_like(s0)
    y = ret.scan_step(x, f, s0, form=c["form"], gate=g, state_out=put)
    up = lambda t: None if t is None else host(t)[:, None]  # noqa: E731
    b_y, b_h, h, _ = scan_bounds(up(x), up(f), c["form"], c["dt"], up(g), host(s0))
    want, _ = oracle.scan(up(x), up(f), c["form"], up(g), host(s0))
    assert within(host(y), want[:, 0], b_y[:, 0]) <= 1
    assert within(host(put), h[:, 0], b_h[:, 0]) <= 1
    y2 = ret.scan_step(x, f, s0, form=c["form"], gate=g)          # in place
    assert torch.equal(y, y2) and torch.equal(s0, put)


def test_steps_continue_a_prefill(torch, ret):
    c = case("bf16", "logit", 2, 200, 96, gate=True, state=True)
    d, x, f, g, s0 = scan_inputs(torch, c, seed=4)
    b_y, b_h, h, _ = scan_bounds(host(x), host(f), "logit", "bf16", host(g), host(s0))
    want, _ = oracle.scan(host(x), host(f), "logit", host(g), host(s0))
    y, s = ret.scan(x[:, :150], f[:, :150], gate=g[:, :150], state_in=s0, state_out=s0.clone())
    assert within(host(y), want[:, :150], b_y[:, :150]) <= 1
    for t in range(150, 200):
        yt = ret.scan_step(x[:, t], f[:, t], s, gate=g[:, t])
        assert within(host(yt), want[:, t], b_y[:, t]) <= 1
    assert within(host(s), h[:, -1], b_h[:, -1]) <= 1


@pytest.mark.parametrize("D", [24, 33])
def test_scan_layouts(torch, ret, D):
    """Spans of a longer sequence, time-major tensors and slices of one buffer give
    what dense copies give, in both directions."""
    d = Draws(torch, "bf16", 10)
    B, N = 3, 270
    buf = d.normal(N, B, 2 * D)                            # time-major, x and f side by side
    x, f = buf[..., :D].transpose(0, 1), buf[..., D:].transpose(0, 1)
    g = d.normal(B, 2 * N, D)[:, 100:100 + N]              # a span of each batch row
    y, cs = ret.scan(x, f, gate=g, return_chunk_states=True)
    dense = [t.contiguous() for t in (x, f, g)]
    want, cs2 = ret.scan(dense[0], dense[1], gate=dense[2], return_chunk_states=True)
    assert torch.equal(y, want) and torch.equal(cs, cs2)
    y2 = torch.empty(N, B, D, device="cuda", dtype=x.dtype).transpose(0, 1)
    ret.scan(x, f, gate=g, out=y2)
    assert torch.equal(y2, want)
    d_y = d.normal(B, 2 * N, D)[:, ::2]                    # every other token
    grads = torch.zeros(N, B, 3 * D, device="cuda", dtype=x.dtype).transpose(0, 1)
    ret.scan_backward(x, f, cs, d_y, gate=g, grad_x=grads[..., :D], grad_f=grads[..., D:2 * D],
                      grad_gate=grads[..., 2 * D:])
    want = ret.scan_backward(dense[0], dense[1], cs, d_y.contiguous(), gate=dense[2])
    assert all(torch.equal(grads[..., k * D:k * D + D], want[k]) for k in range(3))
    with pytest.raises(ret.RetentionError):                # rows that share elements
        ret.scan(x[:1].expand(B, N, D), f)


def test_scan_state_in_place_and_empty(torch, ret):
    d = Draws(torch, "bf16", 5)
    x = d.normal(2, 0, 24)
    s = d.f32(2, 24)
    y, out = ret.scan(x, x, state_in=s, return_state=True)
    assert y.shape == (2, 0, 24) and torch.equal(out, s)
    y, out = ret.scan(x, x, return_state=True)
    assert not out.any()
    gx, gf, gg, ds = ret.scan_backward(x, x, torch.empty(2, 0, 24, device="cuda"), x, gate=x,
                                       d_state_out=s)
    assert torch.equal(ds, s) and gx.shape == x.shape and gg.shape == x.shape
    x, f = d.normal(2, 300, 24), -d.normal(2, 300, 24).abs()
    y, want = ret.scan(x, f, state_in=s, return_state=True)
    ret.scan(x, f, state_in=s, state_out=s)
    assert torch.equal(s, want)


def test_scan_special_values(torch, ret):
    """f of +-inf in both directions, an infinite input behind a reset, NaN in one
    channel only."""
    d = Draws(torch, "f32", 6)
    B, N, D = 1, 200, 40
    for form in ("logit", "log"):
        x, f = d.normal(B, N, D), -d.normal(B, N, D).abs()
        f[:, 90] = -np.inf
        if form == "logit":
            f[:, 120, :7] = np.inf                     # keeps everything, takes nothing
        x[:, 20, 3] = np.nan
        y, s = ret.scan(x, f, form=form, return_state=True)
        want, h = oracle.scan(host(x), host(f), form)
        assert np.isnan(host(y)[0, 20:, 3]).all()
        ok = np.arange(D) != 3
        b_y, _, _, _ = scan_bounds(host(x)[..., ok], host(f)[..., ok], form, "f32")
        assert within(host(y)[..., ok], want[..., ok], b_y) <= 1


def test_scan_leaves_neighbours_alone(torch, ret):
    """Rows and channels around a strided output keep their values."""
    d = Draws(torch, "bf16", 7)
    x, f = d.normal(2, 150, 24), d.normal(2, 150, 24)
    buf = torch.full((2 * 150 + 8, 72), 5.0, device="cuda", dtype=torch.bfloat16)
    out = buf[4:304].view(2, 150, 72)[..., 24:48]
    y = ret.scan(x, f)
    ret.scan(x, f, out=out)
    assert torch.equal(out, y)
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[4:304, 24:48] = False
    assert (buf[mask] == 5).all()


@pytest.mark.parametrize("N,D", [(1000, 128), (5000, 128), (5000, 131)])
def test_scan_streams_and_graphs(torch, ret, N, D):
    """Calls on several streams at once, and a captured pair of calls replayed on new
    inputs: in whole pieces, and dealt over the blocks of a cooperative launch."""
    c = case("bf16", "logit", 2, N, D, gate=True, state=True)
    _, x, f, g, s0 = scan_inputs(torch, c, seed=8)
    want = ret.scan(x, f, gate=g, state_in=s0, return_state=True, return_chunk_states=True)
    d_y = Draws(torch, "bf16", 9).normal(2, N, D)
    back = ret.scan_backward(x, f, want[2], d_y, gate=g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(ret.scan(x, f, gate=g, state_in=s0, return_state=True,
                                    return_chunk_states=True))
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    x2 = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, s, cs = ret.scan(x2, f, gate=g, state_in=s0, return_state=True,
                            return_chunk_states=True)
        grads = ret.scan_backward(x2, f, cs, d_y, gate=g)
    for scale in (1.0, 0.5):
        x2.copy_(x * scale)
        graph.replay()
        torch.cuda.synchronize()
        if scale == 1.0:
            assert torch.equal(y, want[0]) and torch.equal(s, want[1])
            assert all(torch.equal(a, b) for a, b in zip(grads, back))
        else:
            assert torch.equal(y, ret.scan(x2, f, gate=g, state_in=s0))


def test_scan_graphs_share_a_workspace(torch, ret):
    """Two captured calls and an eager one use the same workspace in turn."""
    c = case("f32", "log", 1, 4000, 96, state=True)
    _, x, f, _, s0 = scan_inputs(torch, c, seed=10)
    ws = torch.empty(ret.scan_workspace_bytes(1, 4000, 96, x.dtype), device="cuda",
                     dtype=torch.uint8)
    assert ws.numel() > 0
    want, half = ret.scan(x, f, form="log", state_in=s0), ret.scan(0.5 * x, f, form="log")
    graphs, outs = [], []
    xs = [x.clone(), 0.5 * x]
    for xi, s in zip(xs, (s0, None)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(ret.scan(xi, f, form="log", state_in=s, workspace=ws))
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()
        eager = ret.scan(x, f, form="log", state_in=s0, workspace=ws)
        graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], half) and torch.equal(eager, want)


def test_scan_offsets_past_32_bits(torch, ret):
    """Batch rows more than 2^32 bytes apart, read and written."""
    N, D, far = 300, 64, (1 << 31) + 64
    d = Draws(torch, "bf16", 11)
    room = [torch.empty(far + N * D, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    x, y = (r.as_strided((2, N, D), (far, D, 1)) for r in room)
    x.copy_(d.normal(2, N, D))
    f = forget(d, "logit", 2, N, D, False)
    assert torch.equal(ret.scan(x, f, out=y), ret.scan(x.contiguous(), f))
    _, cs = ret.scan(x, f, return_chunk_states=True)
    d_y = d.normal(2, N, D)
    got = ret.scan_backward(x, f, cs, d_y, grad_f=y)
    want = ret.scan_backward(x.contiguous(), f, cs, d_y)
    assert all(torch.equal(a, b) for a, b in zip(got, want) if a is not None)


# --- norm and gate ----------------------------------------------------------------

NORM_GATE = [
    # dt, B, H, N, dv, norm, gate, token_major
    ("bf16", 1, 1, 1, 8, "layer", True, False), ("f32", 2, 3, 5, 32, "rms", True, True),
    ("bf16", 2, 3, 37, 64, "layer", True, True), ("bf16", 1, 2, 9, 40, "rms", False, True),
    ("bf16", 3, 2, 33, 264, "layer", True, False), ("f32", 1, 3, 17, 264, "layer", True, True),
    ("bf16", 2, 8, 50, 256, "layer", True, True), ("bf16", 1, 4, 30, 512, "rms", True, True),
    ("f32", 1, 2, 7, 512, "layer", False, False), ("bf16", 1, 1, 11, 1024, "layer", True, True),
    ("f32", 1, 2, 5, 1024, "rms", True, True), ("f32", 2, 2, 70, 16, "layer", True, False),
    ("bf16", 1, 5, 19, 128, "layer", True, True),
]


def norm_gate_inputs(torch, c, seed, slices=False):
    dt, B, H, N, dv, norm, gate, tm = c
    d = Draws(torch, dt, seed)
    y = d.rng.standard_normal((B, H, N, dv)) * np.exp(d.rng.standard_normal((B, H, N, 1)))
    y += 2.0 * d.rng.standard_normal((B, H, N, 1))
    if N > 4:
        y[:, :, 3] = 0.0                              # a row of zeros
    shape = (B, N, H, dv) if tm else (B, H, N, dv)
    g = 3 * d.normal(*shape) if gate else None
    if g is not None and tm and slices:               # the gate as a slice of a projection
        p = torch.zeros(B, N, 3 * H * dv, device="cuda", dtype=g.dtype)
        p[..., H * dv:2 * H * dv] = g.reshape(B, N, H * dv)
        g = p[..., H * dv:2 * H * dv].unflatten(-1, (H, dv))
    return d, d.put(y), g, shape


@pytest.mark.parametrize("c", NORM_GATE, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("slices", [False, True])
def test_norm_gate(torch, ret, c, slices):
    dt, B, H, N, dv, norm, gate, tm = c
    d, y, g, shape = norm_gate_inputs(torch, c, 11, slices)
    o = ret.norm_gate(y, g, norm=norm, eps=EPS, token_major=tm)
    want = oracle.norm_gate(host(y), opt(g), norm, EPS, tm)
    e = norm_bound(host(y), norm, EPS)
    e = np.swapaxes(e, 1, 2) if tm else e
    if g is not None:
        gh = host(g)
        e = e * np.abs(gh / (1 + np.exp(-gh))) + (24 + 2.4 * np.abs(gh)) * U * np.abs(want)
    assert o.shape == shape
    assert within(host(o), want, store(dt) * np.abs(want) + e + 1e-37) <= 1


@pytest.mark.parametrize("c", NORM_GATE, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("slices", [False, True])
def test_norm_gate_backward(torch, ret, c, slices):
    dt, B, H, N, dv, norm, gate, tm = c
    d, y, g, shape = norm_gate_inputs(torch, c, 12, slices)
    d_o = d.normal(*shape)
    gy, gg = ret.norm_gate_backward(y, g, d_o, norm=norm, eps=EPS, token_major=tm)
    wy, wg = oracle.norm_gate_backward(host(y), opt(g), host(d_o), norm, EPS, tm)
    z, r = oracle.norm_rows(host(y), norm, EPS)
    e_z = norm_bound(host(y), norm, EPS)
    dd = host(d_o)
    e_d = np.zeros_like(dd)
    if g is not None:
        gh = host(g)
        sig = 1 / (1 + np.exp(-gh))
        slope = sig + gh * sig * (1 - sig)
        zt, e_t = (np.swapaxes(a, 1, 2) if tm else a for a in (z, e_z))
        b = store(dt) * np.abs(wg) + np.abs(dd) * (
            e_t * np.abs(slope) + np.abs(zt) * (28 + 2.4 * np.abs(gh)) * U * (1 + np.abs(gh)))
        assert within(host(gg), wg, b + 1e-37) <= 1
        dd = dd * gh * sig
        e_d = (24 + 2.4 * np.abs(gh)) * U * np.abs(dd)
    else:
        assert gg is None
    if tm:
        dd, e_d = np.swapaxes(dd, 1, 2), np.swapaxes(e_d, 1, 2)
    b = norm_backward_bound(dd, e_d, z, e_z, r, norm, spread_error(host(y), norm, EPS))
    assert within(host(gy), wy, store(dt) * np.abs(wy) + b + 1e-37) <= 1


def test_norm_gate_equals_the_fused_forward(torch, ret):
    """ret_chunkwise then ret_norm_gate against ret_chunkwise_gated on the oracle's
    scale: both round o once, the two-pass form y as well."""
    d = Draws(torch, "f32", 13)
    q, k, v = (0.1 * d.f32(1, 2, 130, 64) for _ in range(3))
    gam = torch.tensor([0.9, 0.97], device="cuda")
    g = d.f32(1, 2, 130, 64)
    fused = ret.chunkwise(q, k, v, gam, 64, gn_eps=EPS, gate=g)
    y = ret.chunkwise(q, k, v, gam, 64)
    o = ret.norm_gate(y, g, norm="layer", eps=EPS)
    assert oracle.rel_frobenius(host(o), host(fused)) <= 1e-5


def test_norm_gate_in_place(torch, ret):
    c = ("bf16", 2, 3, 21, 96, "layer", True, False)
    d, y, g, shape = norm_gate_inputs(torch, c, 14)
    want = ret.norm_gate(y, g)
    for keep in (y, g):
        out = keep.clone()
        args = (out, g) if keep is y else (y, out)
        assert torch.equal(ret.norm_gate(*args, out=out), want)
    d_o = d.normal(*shape)
    wy, wg = ret.norm_gate_backward(y, g, d_o)
    y2, d2 = y.clone(), d_o.clone()
    gy, gg = ret.norm_gate_backward(y2, g, d2, grad_y=y2, grad_gate=d2)
    assert torch.equal(gy, wy) and torch.equal(gg, wg)
    with pytest.raises(ret.RetentionError):               # token-major output over head-major y
        ret.norm_gate(y, g.transpose(1, 2).contiguous(), token_major=True,
                      out=y.view(2, 21, 3, 96))


def test_norm_gate_offsets_past_32_bits(torch, ret):
    """More than 2^31 elements; the last tokens of the last head are checked."""
    B, H, N, dv = 2, 3, 699_200, 512
    g0 = torch.Generator(device="cuda").manual_seed(1)
    y = torch.randn(B, H, N, dv, device="cuda", dtype=torch.bfloat16, generator=g0)
    assert y.numel() > 1 << 31
    gate = torch.randn(B, N, H, dv, device="cuda", dtype=torch.bfloat16, generator=g0)
    o = ret.norm_gate(y, gate, token_major=True)
    tail = ret.norm_gate(y[-1:, :, -5:].contiguous(), gate[-1:, -5:].contiguous(),
                         token_major=True)
    assert torch.equal(o[-1:, -5:], tail)
    del o
    gy, gg = ret.norm_gate_backward(y, gate, gate, token_major=True)
    ty, tg = ret.norm_gate_backward(y[-1:, :, -5:].contiguous(), gate[-1:, -5:].contiguous(),
                                    gate[-1:, -5:].contiguous(), token_major=True)
    assert torch.equal(gy[-1:, :, -5:], ty) and torch.equal(gg[-1:, -5:], tg)


# --- residual and norms -------------------------------------------------------------

ADD_NORM = [
    # dt, rows, d, post, norm, w, w_post, residual
    ("bf16", 1, 1, None, "rms", True, False, True), ("f32", 3, 7, "rms", "layer", True, True, True),
    ("bf16", 5, 64, "layer", "rms", True, True, True),
    ("bf16", 9, 1000, None, "layer", True, True, True),
    ("bf16", 8, 4096, None, "rms", True, False, True),
    ("bf16", 3, 513, "rms", "rms", False, True, False),
    ("f32", 700, 96, "rms", "rms", True, True, True),
    ("f32", 11, 2001, "rms", "rms", True, True, True),
    ("bf16", 650, 2048, "rms", "layer", True, True, True),
    ("f32", 2, 8192, "layer", "layer", True, True, True),
    ("bf16", 2, 16384, "rms", "rms", True, True, True),
    ("f32", 2, 16384, "rms", "rms", True, True, True),
    ("bf16", 2, 16383, None, "rms", True, True, True),
    ("bf16", 2500, 33, None, "rms", True, True, True),
    ("f32", 1300, 260, "layer", "rms", True, False, True),
    ("bf16", 900, 512, "layer", "layer", True, True, True),
    ("bf16", 1900, 1024, "rms", "layer", True, True, True),
    ("f32", 500, 1024, "layer", "layer", True, True, True),
    ("f32", 450, 4096, "rms", "layer", True, True, True),
    ("bf16", 460, 4096, "layer", "rms", True, True, True),
    ("bf16", 300, 8192, "rms", "rms", True, True, True),
    ("bf16", 301, 6000, None, "layer", True, True, True),
    ("bf16", 500, 4095, "rms", "layer", True, True, True),
    ("bf16", 301, 1001, "layer", "rms", True, False, True),
    ("f32", 400, 8191, "rms", "rms", True, True, True),
    ("bf16", 1300, 301, "layer", "layer", True, True, True),
    ("f32", 333, 1025, None, "rms", False, True, True),
]
ALPHA, BETA = 1.5, 0.7


def add_norm_inputs(torch, c, seed):
    dt, rows, dim, post, norm, w, wp, res = c
    d = Draws(torch, dt, seed)
    x = d.rng.standard_normal((rows, dim)) + 0.5
    if rows > 4:
        x[2] = 0.0
    x = d.put(x)
    r = 3 * d.normal(rows, dim) if res else None
    return d, x, r, 1 + 0.3 * d.f32(dim) if w else None, d.f32(dim) if wp else None


def post_part(x, wp, post):
    """(w_post N_post(x), its bound)."""
    u, e = x, np.zeros_like(x)
    if post is not None:
        u, _ = oracle.norm_rows(x, post, EPS)
        e = norm_bound(x, post, EPS)
    wp = 1.0 if wp is None else wp
    return u * wp, (e + 2 * U * np.abs(u)) * np.abs(wp)


@pytest.mark.parametrize("c", ADD_NORM, ids=lambda c: "-".join(map(str, c)))
def test_add_norm(torch, ret, c):
    dt, rows, dim, post, norm, w, wp, res = c
    d, x, r, w, wp = add_norm_inputs(torch, c, 21)
    got_r, got_y = ret.add_norm(x, r, w, w_post=wp, post_norm=post, norm=norm, alpha=ALPHA,
                                beta=BETA, eps=EPS)
    al, be = float(np.float32(ALPHA)), float(np.float32(BETA))
    want_r, want_y = oracle.add_norm(host(x), opt(r), opt(w), opt(wp), post, norm, al, be, EPS)
    u, e_u = post_part(host(x), opt(wp), post)
    e_r = be * e_u + 3 * U * (np.abs(be * u) + (0 if r is None else np.abs(al * host(r))))
    assert within(host(got_r), want_r, store(dt) * np.abs(want_r) + e_r + 1e-37) <= 1
    # y: the norm of a sum that is itself off by e_r
    z, inv = oracle.norm_rows(want_r, norm, EPS)
    mean = lambda t: t.mean(-1, keepdims=True)  # noqa: E731
    e_y = norm_bound(want_r, norm, EPS) + inv * (
        e_r + mean(e_r) + np.abs(z) * (mean(e_r * np.abs(z)) + mean(np.abs(z)) * mean(e_r)))
    wv = 1.0 if w is None else np.abs(host(w))
    b = store(dt) * np.abs(want_y) + 1.01 * wv * e_y + 4 * U * np.abs(want_y) + 1e-37
    assert within(host(got_y), want_y, b) <= 1


@pytest.mark.parametrize("c", ADD_NORM, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("with_res_grad", [True, False])
def test_add_norm_backward(torch, ret, c, with_res_grad):
    dt, rows, dim, post, norm, w, wp, res = c
    d, x, _, w, wp = add_norm_inputs(torch, c, 22)
    r = 3 * d.normal(rows, dim) + 0.5
    d_y, d_r = d.normal(rows, dim), d.normal(rows, dim) if with_res_grad else None
    got = ret.add_norm_backward(x, r, w, d_y, d_r, w_post=wp, post_norm=post, norm=norm,
                                alpha=ALPHA, beta=BETA, eps=EPS)
    al, be = float(np.float32(ALPHA)), float(np.float32(BETA))
    want = oracle.add_norm_backward(host(x), host(r), opt(w), host(d_y), opt(d_r), opt(wp), post,
                                    norm, al, be, EPS)
    z, inv = oracle.norm_rows(host(r), norm, EPS)
    e_z = norm_bound(host(r), norm, EPS)
    dd = host(d_y) * (1.0 if w is None else host(w))
    e_d = norm_backward_bound(dd, U * np.abs(dd), z, e_z, inv, norm,
                              spread_error(host(r), norm, EPS))
    d_sum = want[1] / al
    e_d = e_d + 2 * U * (np.abs(d_sum) + (0 if d_r is None else np.abs(host(d_r))))
    b_res = store(dt) * np.abs(want[1]) + al * (e_d + U * np.abs(d_sum)) + 1e-37
    assert within(host(got[1]), want[1], b_res) <= 1
    du, e_du = be * d_sum, be * (e_d + U * np.abs(d_sum))
    xh, e_x, rx = host(x), np.zeros((rows, dim)), None
    if post is not None:
        xh, rx = oracle.norm_rows(host(x), post, EPS)
        e_x = norm_bound(host(x), post, EPS)
    dx, e_dx = du, e_du
    if wp is not None:
        dx, e_dx = du * host(wp), (e_du + U * np.abs(du)) * np.abs(host(wp))
    if post is not None:
        e_dx = norm_backward_bound(dx, e_dx, xh, e_x, rx, post, spread_error(host(x), post, EPS))
    assert within(host(got[0]), want[0], store(dt) * np.abs(want[0]) + e_dx + 1e-37) <= 1
    # weight gradients: sums over rows, at most rows/592 + 128 additions after one another
    k = (rows / 592 + 128) * U
    if w is not None:
        t = np.abs(host(d_y) * z)
        b = k * t.sum(0) + (np.abs(host(d_y)) * e_z).sum(0) + 1e-37
        assert within(host(got[2]), want[2], b) <= 1
    else:
        assert got[2] is None
    if wp is not None:
        b = k * np.abs(du * xh).sum(0) + (np.abs(du) * e_x + e_du * np.abs(xh)).sum(0) + 1e-37
        assert within(host(got[3]), want[3], b) <= 1
    else:
        assert got[3] is None
    twice = ret.add_norm_backward(x, r, w, d_y, d_r, w_post=wp, post_norm=post, norm=norm,
                                  alpha=ALPHA, beta=BETA, eps=EPS)
    assert all(torch.equal(a, b) for a, b in zip(got, twice) if a is not None)


@pytest.mark.parametrize("dim", [1000, 1001])
def test_add_norm_in_place_and_empty(torch, ret, dim):
    c = ("bf16", 3700, dim, "rms", "rms", True, True, True)
    d, x, r, w, wp = add_norm_inputs(torch, c, 23)
    kw = dict(w_post=wp, post_norm="rms", norm="rms", alpha=ALPHA, beta=BETA)
    want = ret.add_norm(x, r, w, **kw)
    r2, x2 = r.clone(), x.clone()
    got = ret.add_norm(x2, r2, w, res_out=r2, out=x2, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    d_y, d_r = d.normal(3700, dim), d.normal(3700, dim)
    want = ret.add_norm_backward(x, r, w, d_y, d_r, **kw)
    dy2, dr2 = d_y.clone(), d_r.clone()
    got = ret.add_norm_backward(x, r, w, dy2, dr2, grad_x=dy2, grad_residual=dr2, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    none = torch.empty(0, dim, device="cuda", dtype=torch.bfloat16)
    assert ret.add_norm(none, none, w)[1].shape == (0, dim)
    got = ret.add_norm_backward(none, none, w, none, w_post=wp)
    assert not got[2].any() and not got[3].any()


def test_add_norm_offsets_past_32_bits(torch, ret):
    """More than 2^31 elements; the last rows are checked."""
    rows, dim = 1_050_000, 2048
    g0 = torch.Generator(device="cuda").manual_seed(2)
    x, r = (torch.randn(rows, dim, device="cuda", dtype=torch.bfloat16, generator=g0)
            for _ in range(2))
    assert x.numel() > 1 << 31
    w = torch.rand(dim, device="cuda", generator=g0)
    kw = dict(w_post=w, post_norm="rms", norm="layer", alpha=ALPHA, beta=BETA)
    got = ret.add_norm(x, r, w, **kw)
    want = ret.add_norm(x[-7:].clone(), r[-7:].clone(), w, **kw)
    assert all(torch.equal(a[-7:], b) for a, b in zip(got, want))
    del got
    got = ret.add_norm_backward(x, r, w, r, x, **kw)
    want = ret.add_norm_backward(x[-7:].clone(), r[-7:].clone(), w, r[-7:].clone(),
                                 x[-7:].clone(), **kw)
    assert all(torch.equal(a[-7:], b) for a, b in zip(got[:2], want[:2]))


# --- a run of them together ---------------------------------------------------------

def test_block_forward_and_gradients(torch, ret):
    """Two layers as a model runs them: norm, projections, retention, norm and gate,
    projection, residual and norm, gated recurrence, projection, residual and norm;
    gradients of every parameter against torch's float64 autograd of the formulas.
    float32 throughout; each call is within 1e-5, six calls follow one another in
    each direction and no norm here stretches an error more than tenfold."""
    B, N, M, H, dk = 2, 150, 64, 2, 32
    F = torch.nn.functional
    rng = torch.Generator().manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=rng, dtype=torch.float64)  # noqa: E731
    P = dict(wq=mk(M, M) / 8, wk=mk(M, M) / 8, wv=mk(M, M) / 8, wg=mk(M, M) / 8, wo=mk(M, M) / 8,
             wp=mk(M, 3 * M) / 8, w2=mk(M, M) / 8, n1=1 + 0.1 * mk(M), n2=1 + 0.1 * mk(M),
             n3=1 + 0.1 * mk(M))
    P = {k: v.float().double().requires_grad_() for k, v in P.items()}
    x0, c = mk(B, N, M).float().double(), mk(B, N, M).float().double()
    gam = torch.tensor([0.9, 0.97], dtype=torch.float64)

    def rms(v, w):
        return v / (v.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w

    heads = lambda t: t.view(B, N, H, dk).transpose(1, 2)  # noqa: E731
    r = x0
    a = rms(r, P["n1"])
    q, k, v = (heads(a @ P[n]) for n in ("wq", "wk", "wv"))
    i = torch.arange(N, dtype=torch.float64)
    diff = i[:, None] - i[None, :]
    D = torch.where(diff >= 0, gam[:, None, None] ** diff.clamp(min=0), torch.zeros(()).double())
    o = ((q @ k.transpose(-1, -2)) * D) @ v
    z = (o - o.mean(-1, keepdim=True)) / (o.var(-1, unbiased=False, keepdim=True) + EPS).sqrt()
    o = z.transpose(1, 2).reshape(B, N, M) * F.silu(a @ P["wg"])
    r = r + 0.5 * (o @ P["wo"])
    a = rms(r, P["n2"])
    xs, f, g = (a @ P["wp"]).split(M, -1)
    h, hs = torch.zeros(B, M, dtype=torch.float64), []
    for t in range(N):
        s = torch.sigmoid(f[:, t])
        h = s * h + (1 - s) * xs[:, t]
        hs.append(h)
    u = torch.stack(hs, 1) * F.silu(g)
    r = r + 0.5 * (u @ P["w2"])
    y = rms(r, P["n3"])
    (y * c).sum().backward()

    dev = {k: v.detach().float().cuda() for k, v in P.items()}
    X, C, G = x0.float().cuda(), c.float().cuda(), gam.float().cuda()
    flat = lambda t: t.reshape(B * N, -1)  # noqa: E731
    grad = {}
    zero = torch.zeros_like(X)
    r0, a1 = ret.add_norm(zero, X, dev["n1"], eps=EPS)
    Q, K, V = (heads(a1 @ dev[n]).contiguous() for n in ("wq", "wk", "wv"))
    Gt = (a1 @ dev["wg"]).view(B, N, H, dk)
    O = ret.chunkwise(Q, K, V, G, 64)
    og = ret.norm_gate(O, Gt, eps=EPS, token_major=True)
    b1 = og.view(B, N, M) @ dev["wo"]
    r1, a2 = ret.add_norm(b1, r0, dev["n2"], beta=0.5, eps=EPS)
    p = a2 @ dev["wp"]
    px, pf, pg = p.split(M, -1)
    u2, cs = ret.scan(px, pf, gate=pg, return_chunk_states=True)
    b2 = u2 @ dev["w2"]
    r2, y2 = ret.add_norm(b2, r1, dev["n3"], beta=0.5, eps=EPS)

    d_b2, d_r1, grad["n3"], _ = ret.add_norm_backward(b2, r2, dev["n3"], C, None, beta=0.5,
                                                      eps=EPS)
    grad["w2"] = flat(u2).T @ flat(d_b2)
    d_u = d_b2 @ dev["w2"].T
    d_p = torch.empty_like(p)
    ret.scan_backward(px, pf, cs, d_u, gate=pg, grad_x=d_p[..., :M], grad_f=d_p[..., M:2 * M],
                      grad_gate=d_p[..., 2 * M:])
    grad["wp"] = flat(a2).T @ flat(d_p)
    d_b1, d_r0, grad["n2"], _ = ret.add_norm_backward(b1, r1, dev["n2"], d_p @ dev["wp"].T, d_r1,
                                                      beta=0.5, eps=EPS)
    grad["wo"] = flat(og).T @ flat(d_b1)
    d_og = (d_b1 @ dev["wo"].T).view(B, N, H, dk)
    d_O, d_Gt = ret.norm_gate_backward(O, Gt, d_og, eps=EPS, token_major=True)
    dq, dk_, dv_, _ = ret.chunkwise_backward(Q, K, V, G, 64, d_O)
    rows = lambda t: t.transpose(1, 2).reshape(B, N, M)  # noqa: E731
    d_a1 = zero.clone()
    for n, t in (("wq", rows(dq)), ("wk", rows(dk_)), ("wv", rows(dv_)),
                 ("wg", d_Gt.reshape(B, N, M))):
        grad[n] = flat(a1).T @ flat(t)
        d_a1 += t @ dev[n].T
    _, _, grad["n1"], _ = ret.add_norm_backward(zero, r0, dev["n1"], d_a1, d_r0, eps=EPS)
    assert oracle.rel_frobenius(host(y2), y.detach().numpy()) <= 1e-4
    for n, t in P.items():
        assert oracle.rel_frobenius(host(grad[n]), t.grad.numpy()) <= 1e-4, n
