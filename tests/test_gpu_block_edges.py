"""Calls around a linear that the documentation allows and that are easy to get wrong:
statuses that meet, inputs and outputs in one place, bit patterns that no arithmetic
gives, blocks that take several passes, objects that outlive what they were made with."""
import pytest
import torch

from test_gpu_block import packed
from test_gpu_kv_append import Batch
from w4a4_rank_assisted_b200 import hsq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def test_a_timeout_and_a_bad_page_are_both_reported():
    layer = packed(24, 512, 256, 1)
    x, y = torch.randn(24, 512, device=DEV).to(BF), torch.empty(24, 256, device=DEV, dtype=BF)
    b = Batch([4], [0], 8, 2, 4, 128, BF, BF)
    b.table[0, 0] = -1
    append = lambda: hsq.hsq_kv_append(b.k, b.v, b.kc, b.vc, b.table, b.lens_t, cu_seqlens=b.cu)  # noqa: E731
    for order in (0, 1):
        if order:
            append()
        hsq.hsq_debug_force_timeout(1, 30)  # the producer issues nothing: the waits run out after 30 ms
        hsq.forward_x(layer, x, y, layer.workspace_x(24))
        if not order:
            append()
        assert hsq.hsq_get_device_status() == hsq.HSQ_ERR_TIMEOUT
        assert hsq.hsq_get_device_status() == hsq.HSQ_ERR_BAD_PAGE
        assert hsq.hsq_get_device_status() == hsq.HSQ_OK
