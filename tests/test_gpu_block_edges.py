"""Calls around a linear that the documentation allows and that are easy to get wrong:
statuses that meet, inputs and outputs in one place, bit patterns that no arithmetic
gives, blocks that take several passes, objects that outlive what they were made with."""
import pytest
import torch

from test_gpu_epilogue import SHAPES, Layer
from test_gpu_kv_append import Batch, run_and_check
from test_gpu_rope import angles, check, rotate64
from w4a4_rank_assisted_b200 import hsq
from w4a4_rank_assisted_b200.synth import LayerSpec, make_layer

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


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


def _nans(t, seed):
    """Fill a bf16 or fp32 tensor with bit patterns, NaN of every kind among them (an integer view writes them)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    bits = t.view(torch.int16 if t.dtype == BF else torch.int32)
    bits.copy_(torch.randint(-(1 << 15), 1 << 15, t.shape, generator=g, device=DEV) if t.dtype == BF
               else torch.randint(-(1 << 31), 1 << 31, t.shape, generator=g, device=DEV))
    some = ([0x7FC1, 0xFF81 - 0x10000, 0x7F81, -1, 0x7FFF, 0x7F80, 0xFF80 - 0x10000] if t.dtype == BF else
            [0x7FC00001, 0x7F800001, -1, 0x7F800000, -(1 << 23)])
    bits[..., :len(some)] = torch.tensor(some, device=DEV, dtype=bits.dtype)
    bits[..., -len(some):] = torch.tensor(some, device=DEV, dtype=bits.dtype)
    return t


def _same_bits(a, b):
    kind = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,pairs,off", [(64, 16, 0), (72, 4, 0), (64, 16, 1), (31, 7, 0)],
                         ids=["16-byte", "8-byte", "off", "odd"])
@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
def test_what_is_only_moved_keeps_its_bits(dtype, D, pairs, off, adjacent):
    """Elements behind the pairs, values, and heads without a rotation are copied bit for bit, every NaN's sign and
    payload included, in place and out of place, in pieces of any width."""
    T, q, kv, page = 9, 4, 2, 4
    n = T * (q + 2 * kv) * D
    qkv = _nans(torch.empty(n + 8, device=DEV, dtype=dtype)[off:n + off].view(T, q + 2 * kv, D), D)
    freqs = torch.linspace(1.0, 0.1, pairs, device=DEV)
    rot, pos = hsq.Rotation(freqs, interleaved=adjacent), torch.arange(T, device=DEV)
    x, y = qkv[:, :q], torch.zeros(T, q, D, device=DEV, dtype=dtype)
    hsq.hsq_rope(x, y, pos, rot)
    assert _same_bits(y[..., 2 * pairs:], x[..., 2 * pairs:])
    w = qkv.clone()
    hsq.hsq_rope(w[:, :q], w[:, :q], pos, rot)
    assert _same_bits(w[..., 2 * pairs:], qkv[..., 2 * pairs:]) and _same_bits(w[:, q:], qkv[:, q:])
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device=DEV)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    at = torch.arange(T, device=DEV)
    pages, slots = table[0, at // page].long(), at % page
    k, v = qkv[:, q:q + kv], qkv[:, q + kv:]
    for r in (rot, None):
        p = 0 if r is None else 2 * pairs
        kc, vc = (torch.zeros(4, page, kv, D, device=DEV, dtype=dtype) for _ in range(2))
        qo = torch.zeros(T, q, D, device=DEV, dtype=dtype)
        hsq.hsq_kv_append(k, v, kc, vc, table, zero, cu_seqlens=cu, rotation=r, q=x, q_out=qo)
        assert _same_bits(vc[pages, slots], v)
        assert _same_bits(kc[pages, slots][..., p:], k[..., p:]) and _same_bits(qo[..., p:], x[..., p:])
        w = qkv.clone()
        hsq.hsq_kv_append(w[:, q:q + kv], w[:, q + kv:], kc, vc, table, zero, cu_seqlens=cu, rotation=r, q=w[:, :q],
                          q_out=w[:, :q])
        assert _same_bits(w[..., p:], qkv[..., p:]) and _same_bits(w[:, q:], qkv[:, q:])
    if dtype == BF:  # a wider cache holds the same NaN: its upper half
        vc = torch.zeros(4, page, kv, D, device=DEV)
        hsq.hsq_kv_append(k, v, vc.clone(), vc, table, zero, cu_seqlens=cu)
        assert torch.equal(vc[pages, slots].contiguous().view(torch.int32) >> 16, v.contiguous().view(torch.int16).int())


# A block takes a second pass from 18 blocks per SM on (2664 on 148 SMs).  (tokens, heads, dim, pairs, adjacent): 33
# heads of 128 are one block of a token in bf16 and two in fp32, five heads of 511 single elements' units are three,
# whose threads walk over two units each.
MANY = [(6001, 33, 128, 64, False), (6001, 33, 128, 64, True), (5401, 33, 128, 32, False), (1999, 5, 511, 3, True),
        (1999, 5, 511, 3, False)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", MANY, ids=lambda c: "-".join(map(str, c)))
def test_rotation_in_several_passes(case, dtype):
    T, H, D, P, adjacent = case
    g = torch.Generator().manual_seed(T)
    freqs = (100.0 ** (-torch.arange(P, dtype=torch.float64) / P)).float().to(DEV)
    axes = torch.arange(P) % 2
    wide = torch.randn(T, H + 1, D, generator=g).to(dtype).to(DEV)
    x = wide[:, :H]
    pos = torch.randint(0, 5000, (T, 2), generator=g).to(DEV)
    rot = hsq.Rotation(freqs, axes.tolist(), interleaved=adjacent, scale=0.75)
    y = torch.full((T, H, D), float("nan"), device=DEV, dtype=dtype)
    hsq.hsq_rope(x, y, pos, rot)
    want, m = rotate64(x, angles(pos, freqs, axes), adjacent, False, 0.75)
    check(y, want, m, str(case))
    assert torch.equal(y[..., 2 * P:], x[..., 2 * P:])
    w = wide.clone()
    hsq.hsq_rope(w[:, :H], w[:, :H], pos, rot)
    assert torch.equal(w[:, :H], y) and torch.equal(w[:, H:], wide[:, H:])


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (BF, torch.float8_e4m3fn), (F32, BF), (BF, F32)],
                         ids=["bf16", "e4m3", "f32-bf16", "bf16-f32"])
@pytest.mark.parametrize("big", [True, False], ids=["128", "511"])
def test_append_in_several_passes(big, dtype, cache):
    """Ragged prompts whose tokens end inside a block's passes, padding in front and behind, an inactive sequence."""
    q, kv, D, P, real = (32, 8, 128, 64, 6001) if big else (2, 2, 511, 3, 2101)
    lens = [3, 77, -1, 0, 250, 16]
    n = [real // 7, 0, real // 5, 1, real // 3]
    n.append(real - sum(n))
    f = (100.0 ** (-torch.arange(P, dtype=torch.float64) / P)).float().to(DEV)
    scale = [0.02 + 0.1 * torch.rand(kv, device=DEV) for _ in range(2)] if cache == torch.float8_e4m3fn else [None, None]
    for rot, inplace, adjacent in ((hsq.Rotation(f), False, False), (hsq.Rotation(f, interleaved=True), True, True),
                                   (None, False, False)):
        b = Batch(n, lens, 16, kv, q, D, dtype, cache, "heads" if inplace else "slots", pad=5, seed=real, first=2)
        run_and_check(b, rot, f, adjacent, k_scale=scale[0], v_scale=scale[1], q_in_place=inplace)


@pytest.mark.parametrize("i", range(len(SHAPES)), ids=lambda i: "-".join(map(str, SHAPES[i])))
def test_an_epilogue_rounds_once_and_repeats(i):
    """bf16 outputs are the fp32 outputs of the same call rounded once, and every repetition has the same bits."""
    form, fmt, M, K, N, r, group = SHAPES[i]
    lay = Layer(M, K, N, r, group, fmt, seed=i)
    ep = hsq.Epilogue("silu", mul=torch.randn(M, N, device=DEV).to(BF), residual=torch.randn(M, N, device=DEV))
    full, half = torch.empty(M, N, device=DEV), torch.empty(M, N, device=DEV, dtype=BF)
    lay(form, full, ep)
    lay(form, half, ep)
    assert torch.equal(half, full.to(BF))
    for Y in (full, half) * 5:
        want = Y.clone()
        Y.fill_(float("nan"))
        lay(form, Y, ep)
        assert torch.equal(Y, want)


def test_a_long_stream_with_an_epilogue_rounds_once_and_repeats():
    """One token, K = 4096, N = 12288: all SMs, several weight stages a block; among other launches and on its own."""
    lay = Layer(1, 4096, 12288, 4, 64, seed=5, bias=False)
    ep = hsq.Epilogue("silu", mul=torch.randn(1, 12288, device=DEV).to(BF))
    full, half = torch.empty(1, 12288, device=DEV), torch.empty(1, 12288, device=DEV, dtype=BF)
    lay("fused", full, ep)
    for k in range(200):
        half.fill_(float("nan"))
        if k % 3 == 0:
            torch.cuda.synchronize()
        lay("fused", half, ep)
        assert torch.equal(half, full.to(BF))


@pytest.mark.parametrize("form,M,r,group", [("x", 100, 4, 64), ("codes", 300, 4, 128), ("x", 700, 32, 64), ("codes", 513, 0, 64),
                                            ("x", 3700, 4, 128), ("x", 12, 4, 64)])
def test_an_epilogue_with_the_weights_expanded_copy(form, M, r, group):
    """A layer whose weights were expanded once: the bits of the forward that expands them itself."""
    lay = Layer(M, 512, 520, r, group, seed=M)
    Y, want = (torch.empty(M, 520, device=DEV, dtype=BF) for _ in range(2))
    ep = hsq.Epilogue("gelu_tanh", mul=torch.randn(-(-M // 7), 520, device=DEV), mul_rows=7,
                      residual=torch.randn(M, 520, device=DEV).to(BF))
    lay(form, want, ep)
    lay.pl.expand()
    lay(form, Y, ep)
    assert torch.equal(Y, want)


def test_append_with_several_axes_and_no_positions():
    """Every axis then takes the token's place: the bits of one axis."""
    f = torch.linspace(1.0, 0.01, 32, device=DEV)
    out = []
    for axes in (None, [0] * 10 + [1] * 11 + [3] * 11):
        b = Batch([9, 14], [3, 40], 16, 2, 6, 64, BF, BF, pad=2)
        run_and_check(b, hsq.Rotation(f, axes), f)
        out.append((b.kc, b.vc, b.q_out))
    assert all(torch.equal(x, y) for x, y in zip(*out))


def test_append_through_a_column_range_of_a_wider_table():
    """Rows of the block table further apart than their entries; cached lengths and starts inside longer vectors."""
    b = Batch([5, 30, 1], [3, 16, 40], 8, 2, 4, 64, BF, torch.float8_e4m3fn)
    f = torch.linspace(1.0, 0.01, 32, device=DEV)
    wide = torch.full((3, b.table.shape[1] + 6), 1 << 30, dtype=torch.int32, device=DEV)
    wide[:, 5:-1] = b.table
    b.table = wide[:, 5:-1]
    long = torch.full((9,), -7, dtype=torch.int32, device=DEV)
    long[1:4], long[5:] = b.lens_t, b.cu
    b.lens_t, b.cu = long[1:4], long[5:]
    run_and_check(b, hsq.Rotation(f), f)
