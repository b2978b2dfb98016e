"""Calls of the paged serving operators that are refused on the host, or decided there, without a GPU."""
import pytest
import torch

import paged_attention_varlen_b200 as ala


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_attention_varlen_b200 import build
    build.build()


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _aligned(*shape, dtype=torch.bfloat16):
    n = 1
    for s in shape:
        n *= s
    buf = torch.zeros(n + 64, dtype=dtype)
    at = -(buf.data_ptr() % 64) % 64 // buf.element_size()
    return buf[at:at + n].view(shape)


# ---------------------------------------------------------------------------------------------- host tensors

class _Stream:
    cuda_stream = 0


def _cpu_calls():
    """The four planned calls over tensors in host memory (planning them is allowed)."""
    q, kc = _aligned(3, 4, 64), _aligned(6, 16, 2, 64)
    yield ala.plan_paged_step(_i32(3), _i32(3), _i32(3, 4), _i32(6), _i32(1), 16, 5)[0]
    yield ala.plan_paged_write(q[:, :2], None, _i32(3), kc, None)
    yield ala.plan_paged_attention(q, kc, kc, _i32(3, 4), _i32(3), _i32(3), 9, 4, 2, 0.125)[0]
    yield ala.plan_paged_diff_attention(_aligned(3, 4, 32), _aligned(6, 16, 2, 32), _aligned(6, 16, 1, 64), _i32(3, 4), _i32(3), _i32(3),
                                        torch.zeros(2), 9, 2, 1, 0.125)[0]


@pytest.mark.parametrize("stream", [None, _Stream()])
@pytest.mark.parametrize("which", range(4))
def test_calls_over_host_tensors_launch_nothing(which, stream, monkeypatch):
    launched = []

    def stub(*args):
        launched.append(args)
        return 0

    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    call = list(_cpu_calls())[which]
    setattr(call, "_function" if isinstance(call, ala.PagedCall) else "_execute", stub)
    with pytest.raises(ValueError):
        call(stream)
    assert not launched
