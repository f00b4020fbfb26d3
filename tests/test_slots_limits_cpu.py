"""Limits of the slot calls' sizes and strides, on a host without a GPU: what passes every check ends
with the launch's own error there (HIP), what does not with UNSUPPORTED."""
import ctypes

import pytest
import torch

import quantized_recurrent_state_amd as lsq
from quantized_recurrent_state_amd import _lib
from tests.test_slots_cpu import batch, handle

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="its made-up addresses must not reach a GPU")
UNSUPPORTED, HIP = 2, 5


def attend(h, **kw):
    return _lib.load().lsq_attend(h, ctypes.byref(batch(**kw)), None, 0, None)


def test_a_launch_is_refused_by_its_own_threads():
    # 16-bit types of up to 64 value columns run workgroups of 256 threads, others of 512
    h = handle()                                            # 4 heads, dv 64: 4 workgroups per entry
    for seqs, narrow, wide in ((1 << 21, HIP, UNSUPPORTED), ((1 << 22) - 1, HIP, UNSUPPORTED),
                               (1 << 22, UNSUPPORTED, UNSUPPORTED), ((1 << 21) - 1, HIP, HIP)):
        assert attend(h, seqs=seqs, tokens=100) == narrow, seqs
        assert attend(h, seqs=seqs, tokens=100, io=lsq.IO_F32) == wide, seqs
    lsq.lsq_state_free(h)


@pytest.mark.parametrize("io", [lsq.IO_BF16, lsq.IO_F32])
@pytest.mark.parametrize("name", ["q_stride", "k_stride", "v_stride", "o_stride"])
def test_a_far_stride_is_refused_whatever_its_size(name, io):
    h = handle()
    e = 4 if io == lsq.IO_F32 else 2
    far = (32 << 20) // e                                   # 32 MiB between tokens
    for stride in (far, 1 << 40, 1 << 61, 1 << 62, (1 << 62) + 256, (1 << 63) - 256):
        assert attend(h, tokens=100, io=io, **{name: stride}) == UNSUPPORTED, stride
    assert attend(h, tokens=100, io=io, **{name: far - 8}) == HIP
    lsq.lsq_state_free(h)
