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
