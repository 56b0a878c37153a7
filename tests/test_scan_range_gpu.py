"""The gated linear recurrence at the ends of its stated range: rows of more than
2^31 bytes."""
import pytest

from test_block_gpu import no_device_error, ret, torch  # noqa: F401 (fixtures)

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
