"""GPU tests of what the decode-time products (qlora_fmt4_linear_fwd, qlora_moe_fwd) do at their
edges: waits that run out, the ends of the fp32 range, calls on another stream, refusals."""
import pytest
import torch

import bit_nf4_quantized_double_b200 as q

pytestmark = pytest.mark.gpu


def test_a_warps_wait_has_one_answer():
    # 24 waits that complete, 24 that are aborted, 48 that get both at nearly the same time, one that runs into its limit
    assert q.qlora_get_device_status() == q.QLORA_OK
    out = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    assert q.lib().qlora_selftest_wait_warp(out.data_ptr(), None) == q.QLORA_OK
    assert q.qlora_get_device_status() == q.QLORA_ERR_TIMEOUT
    split, wrong, gave_up, waits = out.tolist()
    assert split == 0 and wrong == 0 and waits == 97
    assert 25 <= gave_up <= 73
