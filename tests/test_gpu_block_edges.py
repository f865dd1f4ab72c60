"""Calls around a linear that the documentation allows and that are easy to get wrong:
statuses that meet, inputs and outputs in one place, bit patterns that no arithmetic
gives, blocks that take several passes, objects that outlive what they were made with."""
import pytest
import torch

from test_gpu_kv_append import Batch
from w4a4_rank_assisted_b200 import hsq
from w4a4_rank_assisted_b200.synth import LayerSpec, make_layer

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def packed(M, K, N, seed, group=64, r=4):
    lay = make_layer(LayerSpec("e", M, K, N, r, act="outlier", outlier_frac=0.01, outlier_mult=5.0, seed=seed, group=group))
    low = (None, None) if r == 0 else (lay.L1.to(DEV), lay.L2.to(DEV))
    return hsq.PackedLinear(lay.W.to(DEV), torch.ones(K, device=DEV), *low, group=group)


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


@pytest.mark.parametrize("M,K,r,group", [(5, 256, 4, 64), (16, 1152, 0, 64), (16, 2048, 4, 128), (3, 512, 8, 64)])
def test_the_decode_tile_form_takes_y_over_x(M, K, r, group):
    """Its grid barrier stands between the last read of X and the first write of Y: without an epilogue, or with one
    that asks for nothing, the bits of a Y of its own; with one it refuses."""
    layer = packed(M, K, K, M, group, r=r)
    assert hsq.hsq_fused_form(M, K, K, r, group) == 2
    x = torch.randn(M, K, device=DEV).to(BF)
    want = torch.empty_like(x)
    hsq.forward_fused(layer, x, want)
    for ep in (None, hsq.Epilogue()):
        for _ in range(5):
            y = x.clone()
            hsq.forward_fused(layer, y, y, epilogue=ep)
            assert torch.equal(y, want)
    with pytest.raises(hsq.HsqError):
        hsq.forward_fused(layer, x, x, epilogue=hsq.Epilogue("relu"))
    assert hsq.hsq_get_device_status() == hsq.HSQ_OK


def test_append_of_as_many_head_blocks_as_a_grid_holds():
    """65534 + 2 * 32768 heads of single elements: 65535 blocks.  Position 0 turns nothing, so all is copied."""
    q, kv, D = 65534, 32768, 511
    qkv = torch.randn(1, q + 2 * kv, D, device=DEV).to(BF)
    kc, vc = torch.zeros(1, 1, kv, D, device=DEV, dtype=BF), torch.zeros(1, 1, kv, D, device=DEV, dtype=BF)
    qo = torch.zeros(1, q, D, device=DEV, dtype=BF)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    hsq.hsq_kv_append(qkv[:, q:q + kv], qkv[:, q + kv:], kc, vc, zero[None], zero, q=qkv[:, :q], q_out=qo,
                      rotation=hsq.Rotation(torch.ones(64, device=DEV)))
    assert torch.equal(qo, qkv[:, :q]) and torch.equal(kc[0, 0], qkv[0, q:q + kv]) and torch.equal(vc[0, 0], qkv[0, q + kv:])
    assert hsq.hsq_get_device_status() == hsq.HSQ_OK
