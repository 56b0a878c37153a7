"""The recurrence where a block works on many items, dealt over the GPU in the order
of time: its ring of items goes round, and the words that blocks publish and look
for are those of a long chain.  Checked against the float64 oracle."""
import os
import re

import pytest

from test_block_gpu import no_device_error, ret, torch  # noqa: F401 (fixtures)
from test_block_gpu import case, ids
from test_block_gpu import test_scan as check_forward
from test_block_gpu import test_scan_backward as check_backward

pytestmark = pytest.mark.gpu

CASES = [
    # rows aligned to 16 bytes, to 4 and to 2; both forms, with a gate and without
    case("bf16", "logit", 1, 16384, 768, state=True, resets=False),
    case("bf16", "log", 2, 8192, 800, gate=True, fused=True, resets=False),
    case("bf16", "log", 1, 12288, 1022, state=True, resets=False),
    case("bf16", "logit", 1, 12288, 1021, gate=True, state=True, resets=False),
    case("f32", "logit", 1, 9000, 700, gate=True, state=True, resets=False),
    case("f32", "log", 3, 5000, 391, state=True, resets=True),
    # more pieces of channels than blocks: an item of a block is in the next turn or this one
    case("f32", "log", 1, 2816, 149 * 32, gate=True, resets=False),
]


def deals(torch, c, which):
    """Asserts that the call is dealt, more items to a block than its ring holds."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    path = os.path.join(root, "linear_recurrent_sequence_scale_b200", "csrc", "scan.cu")
    src = open(path).read()
    constant = lambda name: int(re.search(rf"{name} = (\d+)", src).group(1))  # noqa: E731
    tok = constant("kTokForward" if which == "forward" else "kTokBackward")
    stages = int(re.search(r"kStages = kFit < (\d+)", src).group(1))
    blocks = torch.cuda.get_device_properties(0).multi_processor_count
    pieces = c["B"] * -(-c["D"] // (64 if c["dt"] == "bf16" else 32))
    tiles = -(-c["N"] // tok)
    rounds = tiles * -(-pieces // blocks)        # if blocks kept whole pieces
    assert rounds > constant("kFewRounds") and rounds - 3 > pieces * tiles // blocks
    assert pieces * tiles > stages * blocks


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_many_items_of_a_block_forward(torch, ret, c):
    deals(torch, c, "forward")
    check_forward(torch, ret, c)


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_many_items_of_a_block_backward(torch, ret, c):
    deals(torch, c, "backward")
    check_backward(torch, ret, c)
