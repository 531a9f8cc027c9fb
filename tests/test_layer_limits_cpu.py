"""Limits of the recurrent layer's calls that no launch may pass, checked on
the host with fake device addresses (nothing is launched)."""
import ctypes as C

import pytest

from quantized_recurrent_state_lq_b200 import lq

BASE = 0x7f0000000000
GAP = 1 << 36


def at(i):
    return BASE + i * GAP


@pytest.mark.parametrize("B", [(1 << 30) + 1, (1 << 31) - 2, (1 << 31) - 1])
def test_convolution_refuses_more_sequences_than_its_counters_hold(B):
    """One channel and two taps: a batch that memory would hold, but whose last
    sequence numbers plus a thread's share pass 32 bits."""
    c = lq.lq_conv_config(lq.LQ_BF16, B, 1, 2, lq.LQ_ACT_NONE)
    p = C.addressof(c)
    assert lq.lib().lq_conv_step(p, at(0), at(1), 1, at(2), None, at(3), 1, None) == lq.LQ_ERR_SHAPE
    assert lq.lib().lq_conv_prefill(p, 64, at(4), at(1), 1, at(2), None, None, at(0), at(3), 1, None) == lq.LQ_ERR_SHAPE


def test_wait_selftest_refuses():
    def call(dtype=lq.LQ_BF16, rows=300, row=0, B=1):
        c = lq.lq_ssm_config(dtype, B, 2, 1, 64, 64, 1)
        return lq.lib().lq_selftest_ssm_wait(C.addressof(c), rows, None, at(0), 128, at(1), 2, at(2), at(3), 64, at(4), 64,
                                             None, None, None, at(5), at(6), 128, None, 0, row, None)
    assert call(row=-1) == lq.LQ_ERR_INVALID_ARG and call(row=300) == lq.LQ_ERR_INVALID_ARG
    assert call(dtype=lq.LQ_F32) == lq.LQ_ERR_UNSUPPORTED
    assert call(rows=2000) == lq.LQ_ERR_WORKSPACE      # as in lq_ssm_prefill
    assert call(B=7) == lq.LQ_ERR_SHAPE
