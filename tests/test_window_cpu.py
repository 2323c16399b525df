"""Refusals of the windowed attention calls and of rq_cache_read that need no
GPU: null handles and pointers, and the binding's checks of its tensors."""
import pytest
import torch

import decode_attention_14_b200 as rq


@pytest.mark.parametrize("window,sinks,kind", [(4, 1, 0), (0, 0, 1), (-1, 0, 0), (4, -1, 0), (4, 1, 7)])
def test_null_handles_are_refused(window, sinks, kind):
    assert rq.lib.rq_decode_attn_window(None, 0, 0, None, None, kind, 0.0, window, sinks, None) == rq.RQ_ERR_INVALID
    assert rq.lib.rq_prefill_attn_window(None, 0, 0, None, 3, None, kind, 0.0, window, sinks, None) == rq.RQ_ERR_INVALID
    assert rq.lib.rq_cache_read(None, 0, 0, 0, 1, kind, None, None, 128, 128, 128, None) == rq.RQ_ERR_INVALID


def test_rows_must_be_cuda_tensors_of_a_known_type():
    shape = (1, 2, 3, 128)
    with pytest.raises(ValueError, match="CUDA"):
        rq._check_rows(torch.zeros(shape), shape, "k")
    for dtype in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(ValueError, match="float32 or bfloat16"):
            rq._out_type(dtype)
    assert rq._out_type(torch.float32) == rq.RQ_OUT_FP32 and rq._out_type(torch.bfloat16) == rq.RQ_OUT_BF16


def test_queries_must_be_contiguous_cuda_bfloat16():
    with pytest.raises(ValueError):
        rq._check_dev(torch.zeros((1, 2, 128), dtype=torch.bfloat16), "bfloat16", (1, 2, 128), "q")


@pytest.mark.parametrize("offset,aligned", [(0, True), (1, False), (4, False), (8, True)])
def test_rows_must_be_16_byte_aligned(offset, aligned):
    t = torch.zeros(512, dtype=torch.bfloat16)
    assert t.data_ptr() % 16 == 0
    if aligned:
        rq._check_aligned(t[offset:], "q")
    else:
        with pytest.raises(ValueError, match="16-byte"):
            rq._check_aligned(t[offset:], "q")
