"""A wait of the recurrence that runs out: an error code, never a hang, and the next
call is right.  No GPU fault is involved: the waited-for item is one that no block
works on, and the wait has a short limit."""
import ctypes

import pytest

import linear_recurrent_sequence_scale_b200 as ret

P = ctypes.c_void_p
ROOM = 256 * 1024


def test_scan_wait_selftest_refusals():
    import os
    if not os.path.exists(ret.LIB_PATH):
        from linear_recurrent_sequence_scale_b200 import build
        build.build()
    call = ret.load_library().ret_selftest_scan_wait
    assert call(0, P(0x10000), ROOM, None) == ret.RET_EINVAL
    assert call(10001, P(0x10000), ROOM, None) == ret.RET_EINVAL
    assert call(10, P(0x10008), ROOM, None) == ret.RET_EINVAL
    assert call(10, None, ROOM, None) == ret.RET_EWORKSPACE
    assert call(10, P(0x10000), ROOM - 1, None) == ret.RET_EWORKSPACE


@pytest.mark.gpu
def test_scan_wait_runs_out_and_reports():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib = ret.load_library()
    x, f = (torch.randn(2, 3000, 64, device="cuda") for _ in range(2))
    want = ret.scan(x, f)
    assert ret.device_error() == 0
    room = torch.full((ROOM + 4096,), 7, dtype=torch.uint8, device="cuda")
    stream = P(torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        assert lib.ret_selftest_scan_wait(20, P(room.data_ptr()), ROOM, stream) == ret.RET_OK
        torch.cuda.synchronize()
        assert 801 <= ret.device_error() <= 811
        assert ret.device_error() == 0          # read and cleared
        assert (room[ROOM:] == 7).all()
        y = room[1024 + 2 * 65536:1024 + 3 * 65536].view(torch.float32).view(512, 32)
        assert not y[:256].any()                # the item that nothing worked on
        assert torch.equal(ret.scan(x, f), want)
    assert ret.device_error() == 0
