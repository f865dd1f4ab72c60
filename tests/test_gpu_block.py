"""The calls around a linear as a transformer block runs them: fused QKV linear, cache
append with the rotation (or the rotation alone), attention in plain torch over what
was written, the way back onto the residual stream, a gated MLP.  Each step is
checked from the tensors it was given, so that a rounding does not grow through the
quantizers behind it; then the block is captured and replayed."""
import pytest
import torch

from test_gpu_epilogue import _check, _expect
from test_gpu_rope import check, rotate64
from w4a4_rank_assisted_b200 import hsq
from w4a4_rank_assisted_b200.synth import LayerSpec, make_layer

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def packed(M, K, N, seed, group=64, bias=False):
    lay = make_layer(LayerSpec("b", M, K, N, 4, act="outlier", outlier_frac=0.01, outlier_mult=5.0, seed=seed, bias=bias,
                               group=group))
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    return hsq.PackedLinear(d(lay.W), torch.ones(K, device=DEV), d(lay.L1), d(lay.L2), d(lay.bias), group=group)


def z_of(layer, X, ws):
    """The linear alone, in fp32."""
    z = torch.empty(X.shape[0], layer.N, device=DEV)
    return hsq.forward_x(layer, X, z, ws, out=hsq.HSQ_OUT_F32)


class Block:
    """A decoder block of D = 64 heads over a paged cache, with buffers for T tokens."""

    def __init__(self, T, hidden=256, q=4, kv=2, D=64, mlp=512, pages=24, page=16):
        self.q, self.kv, self.D, self.page = q, kv, D, page
        self.layers = [packed(T, hidden, (q + 2 * kv) * D, 1), packed(T, q * D, hidden, 2), packed(T, hidden, mlp, 3, 128),
                       packed(T, hidden, mlp, 4, 128), packed(T, mlp, hidden, 5, 128)]
        self.ws = [layer.workspace_x(T) for layer in self.layers]
        e = lambda *s: torch.empty(*s, device=DEV, dtype=BF)  # noqa: E731
        self.qkv, self.att, self.up, self.act = e(T, q + 2 * kv, D), e(T, q * D), e(T, mlp), e(T, mlp)
        self.kc, self.vc = (torch.zeros(pages, page, kv, D, device=DEV, dtype=BF) for _ in range(2))
        self.freqs = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().to(DEV)
        self.rot = hsq.Rotation(self.freqs)
        self.gate = hsq.Epilogue("silu", mul=self.up)

    def attention(self, table, lens, cu):
        """Plain torch over the pages, causal; out [T, q * D]."""
        for b, (n, a, e) in enumerate(zip(lens, cu, cu[1:])):
            k, v = (c[table[b].long()].reshape(-1, self.kv, self.D)[:n + e - a].float() for c in (self.kc, self.vc))
            g = self.q // self.kv
            s = torch.einsum("thd,shd->hts", self.qkv[a:e, :self.q].float(), k.repeat_interleave(g, 1)) / self.D ** 0.5
            seen = torch.arange(n + e - a, device=DEV)[None] <= n + torch.arange(e - a, device=DEV)[:, None]
            p = torch.softmax(s.masked_fill(~seen, float("-inf")), -1)
            self.att[a:e] = torch.einsum("hts,shd->thd", p, v.repeat_interleave(g, 1)).reshape(e - a, self.q * self.D).to(BF)

    def project(self, x, table, lens, cu):
        hsq.forward_x(self.layers[0], x, self.qkv.view(x.shape[0], -1), self.ws[0])
        qv = self.qkv[:, :self.q]
        hsq.hsq_kv_append(self.qkv[:, self.q:self.q + self.kv], self.qkv[:, self.q + self.kv:], self.kc, self.vc, table,
                          lens, cu_seqlens=cu, rotation=self.rot, q=qv, q_out=qv)

    def back(self, x):
        hsq.forward_x(self.layers[1], self.att, x, self.ws[1], epilogue=hsq.Epilogue(residual=x))
        hsq.forward_x(self.layers[3], x, self.up, self.ws[3])
        hsq.forward_x(self.layers[2], x, self.act, self.ws[2], epilogue=self.gate)
        hsq.forward_x(self.layers[4], self.act, x, self.ws[4], epilogue=hsq.Epilogue(residual=x))


@pytest.mark.parametrize("new,lens", [([1], [0]), ([1] * 5, [3, 15, 16, 40, 0]), ([30, 1, 0, 70], [2, 16, 9, 0]),
                                      ([300, 57], [0, 11])], ids=["first", "decode", "mixed", "prefill"])
def test_decoder_block_step_by_step(new, lens):
    T = sum(new)
    b = Block(T, pages=40)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    perm = torch.randperm(40).tolist()
    table = torch.tensor([[perm.pop() if j * 16 < a + n else -1 for j in range(24)] for a, n in zip(lens, new)],
                         dtype=torch.int32, device=DEV)
    lens_t, cu_t = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in (lens, cu))
    x0 = torch.randn(T, 256, device=DEV).to(BF)
    x = x0.clone()
    raw = torch.empty_like(b.qkv)
    hsq.forward_x(b.layers[0], x, raw.view(T, -1), b.ws[0])
    b.project(x, table, lens_t, None if new == [1] * len(new) else cu_t)
    at = torch.cat([torch.arange(a, a + n) for a, n in zip(lens, new)]).double()
    want, m = rotate64(raw[:, :6], at[:, None] * b.freqs.cpu().double(), False)
    check(b.qkv[:, :4], want[:, :4], m[:, :4], "q")
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    page, slot = table.cpu()[seq, (at // 16).long()].long(), (at % 16).long()
    check(b.kc.cpu()[page, slot], want[:, 4:], m[:, 4:], "k")
    assert torch.equal(b.vc.cpu()[page, slot], raw[:, 6:].cpu())
    b.attention(table.clamp_min(0), lens, cu)
    z = z_of(b.layers[1], b.att, b.ws[1])
    x1 = x.clone()
    hsq.forward_x(b.layers[1], b.att, x, b.ws[1], epilogue=hsq.Epilogue(residual=x))
    _check(x, *_expect(z, "none", None, 1, x1), "attention residual")
    hsq.forward_x(b.layers[3], x, b.up, b.ws[3])
    hsq.forward_x(b.layers[2], x, b.act, b.ws[2], epilogue=b.gate)
    _check(b.act, *_expect(z_of(b.layers[2], x, b.ws[2]), "silu", b.up, 1, None), "gated MLP")
    z, x2 = z_of(b.layers[4], b.act, b.ws[4]), x.clone()
    hsq.forward_x(b.layers[4], b.act, x, b.ws[4], epilogue=hsq.Epilogue(residual=x))
    _check(x, *_expect(z, "none", None, 1, x2), "MLP residual")
    # the same block as one run of calls, and captured: the same bits
    kc, vc = b.kc.clone(), b.vc.clone()
    y = x0.clone()
    b.project(y, table, lens_t, cu_t)
    b.attention(table.clamp_min(0), lens, cu)
    b.back(y)
    assert torch.equal(y, x) and torch.equal(b.kc, kc) and torch.equal(b.vc, vc)
    att = b.att.clone()
    xg = x0.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.project(xg, table, lens_t, cu_t)
        b.back(xg)
    for _ in range(2):
        xg.copy_(x0)
        b.kc.zero_()
        b.att.copy_(att)
        g.replay()
        assert torch.equal(xg, x)
        assert torch.equal(b.kc.cpu()[page, slot], kc.cpu()[page, slot])
    assert hsq.hsq_get_device_status() == hsq.HSQ_OK


def test_image_block_rotates_q_and_k_of_the_fused_output():
    """Two samples of an image transformer: QKV, one rotation of q and k in place over three axes, the way back with
    a gate per sample, MLP with its GELU; NVFP4 for the way back of the MLP."""
    B, S, heads, D, hidden = 2, 75, 4, 64, 256
    T = B * S
    qkv_l, out_l, up_l = packed(T, hidden, 3 * heads * D, 1, bias=True), packed(T, heads * D, hidden, 2), packed(T, hidden, 1024, 3, bias=True)
    lay = make_layer(LayerSpec("f", T, 1024, hidden, 4, act="outlier", outlier_frac=0.01, outlier_mult=5.0, seed=7, bias=True))
    down_l = hsq.Fp4Linear(lay.W.to(DEV), torch.ones(1024, device=DEV), lay.L1.to(DEV), lay.L2.to(DEV), lay.bias.to(DEV))
    x = torch.randn(T, hidden, device=DEV).to(BF)
    mods = torch.randn(B, 6 * hidden, device=DEV).to(BF)  # a modulation layer's output: gates are column ranges of it
    qkv = torch.empty(T, 3 * heads, D, device=DEV, dtype=BF)
    ws = qkv_l.workspace_x(T)
    hsq.forward_x(qkv_l, x, qkv.view(T, -1), ws)
    raw = qkv.clone()
    ids = torch.stack([torch.zeros(S), torch.arange(S) // 15, torch.arange(S) % 15], 1).to(DEV)
    freqs = torch.cat([100.0 ** (-torch.arange(n, dtype=torch.float64) / n) for n in (4, 14, 14)]).float().to(DEV)
    axes = [0] * 4 + [1] * 14 + [2] * 14
    qk = qkv[:, :2 * heads]
    hsq.hsq_rope(qk, qk, ids, hsq.Rotation(freqs, axes, interleaved=True))
    ang = (ids.cpu().double()[:, axes] * freqs.cpu().double()).repeat(B, 1)
    check(qk, *rotate64(raw[:, :2 * heads], ang, True), "q and k")
    assert torch.equal(qkv[:, 2 * heads:], raw[:, 2 * heads:])
    q, k, v = (t.reshape(B, S, heads, D).float() for t in qkv.split(heads, 1))
    p = torch.softmax(torch.einsum("bthd,bshd->bhts", q, k) / 8, -1)
    att = torch.einsum("bhts,bshd->bthd", p, v).reshape(T, -1).to(BF)
    ws = out_l.workspace_x(T)
    z, x0 = z_of(out_l, att, ws), x.clone()
    hsq.forward_x(out_l, att, x, ws, epilogue=hsq.Epilogue(mul=mods[:, 2 * hidden:3 * hidden], mul_rows=S, residual=x))
    _check(x, *_expect(z, "none", mods[:, 2 * hidden:3 * hidden], S, x0), "gated residual")
    ws, h = up_l.workspace_x(T), torch.empty(T, 1024, device=DEV, dtype=BF)
    hsq.forward_x(up_l, x, h, ws, epilogue=hsq.Epilogue("gelu_tanh"))
    _check(h, *_expect(z_of(up_l, x, ws), "gelu_tanh", None, 1, None), "gelu")
    act, z, x1 = hsq.Fp4ActBuffers(T, 1024, 4, DEV), torch.empty(T, hidden, device=DEV), x.clone()
    hsq.fp4_forward(down_l, h, act, z, out=hsq.HSQ_OUT_F32)
    hsq.fp4_forward(down_l, h, act, x, epilogue=hsq.Epilogue(mul=mods[:, 5 * hidden:], mul_rows=S, residual=x))
    _check(x, *_expect(z, "none", mods[:, 5 * hidden:], S, x1), "NVFP4 gated residual")
    assert hsq.hsq_get_device_status() == hsq.HSQ_OK


@pytest.mark.parametrize("M", [4, 40, 500, 4000])
def test_y_over_x_in_the_one_call_forward(M):
    """The one-call forward may write onto its input (activations are quantized before Y is written); the single launch
    refuses it."""
    layer = packed(M, 256, 256, M)
    ws = layer.workspace_x(M)
    x = torch.randn(M, 256, device=DEV).to(BF)
    want = torch.empty_like(x)
    hsq.forward_x(layer, x, want, ws, epilogue=hsq.Epilogue("gelu_erf", residual=x.clone()))
    y = x.clone()
    hsq.forward_x(layer, y, y, ws, epilogue=hsq.Epilogue("gelu_erf", residual=y))
    assert torch.equal(y, want)
    if M <= 16:
        with pytest.raises(hsq.HsqError):
            hsq.forward_fused(layer, y, y, epilogue=hsq.Epilogue(residual=y))
