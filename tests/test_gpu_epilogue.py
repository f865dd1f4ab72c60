"""The forwards' epilogue act(z) * mul + residual on the GPU.

Reference: z as the forward without an epilogue returns it in fp32 (tested on its
own against the oracle; the accumulation is the same code), the epilogue in fp64
from there.  Tolerance, relative to the value that is rounded, in units of 2^-24
(u; a fast-math bound of n ulp is 2 n u):
  silu, tanh gelu   z / (1 + e^t): e^t to 2 + 1.2 |t| ulp and the argument t to 4 u
                    |t|, both damped by e^t / (1 + e^t); the sum 1 u, the quotient
                    2 ulp: 5 u + (4 + 2.4 |t| + 4 |t|) u
  erf gelu          erfc to 4 ulp, its argument w = |z| / sqrt 2 to 2 u: 2 u (2 w^2 + 1)
                    more; two products: 8 u + 4 u (w^2 + 1) + 2 u
  mul, residual     one rounding each: |act mul| u + |y| u
  the output        half a step: 2^-24 |y| for fp32, 2^-8 |y| for bf16
Values whose e^t overflows are 0 within 2^-100."""
import math

import numpy as np
import pytest
import torch

from _helpers import oracle_layer, rms
from w4a4_rank_assisted_b200 import hsq
from w4a4_rank_assisted_b200.synth import LayerSpec, make_layer

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def _act64(z, act):
    """(act(z), its relative tolerance) in fp64."""
    zero = torch.zeros_like(z)
    if act == "none":
        return z, zero
    if act == "relu":
        return torch.where(z < 0, zero, z), zero
    if act == "gelu_erf":
        w2 = z * z / 2
        return 0.5 * z * torch.special.erfc(-z * math.sqrt(0.5)), (10 + 4 * (w2 + 1)) * U
    t = -z if act == "silu" else -2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    return z * torch.special.expit(-t), (9 + 6.4 * t.abs()) * U


def _expect(z32, act, mul, mul_rows, residual):
    """The epilogue in fp64, and the largest error the arithmetic allows before the output's rounding."""
    z = z32.double()
    y, rel = _act64(z, act)
    tol = y.abs() * rel + 2.0 ** -100
    if mul is not None:
        m = mul.double()[torch.arange(z.shape[0], device=z.device) // mul_rows]
        y, tol = y * m, tol * m.abs()
        tol = tol + y.abs() * U
    if residual is not None:
        y = y + residual.double()
        tol = tol + y.abs() * U
    return y, tol


def _check(Y, y, tol, where):
    half = 2.0 ** -8 if Y.dtype == torch.bfloat16 else 2.0 ** -24
    d = (Y.double() - y).abs()
    bad = ~(d <= tol * (1 + half) + y.abs() * half)
    assert not bad.any(), (f"{where}: {int(bad.sum())} of {bad.numel()} off, worst {float(d.max()):.3e} at "
                           f"{np.unravel_index(int(d.argmax()), d.shape)}, rms {rms(y.cpu().numpy()):.3e}")


class Layer:
    def __init__(self, M, K, N, r, group=64, fmt="int4", seed=0, bias=True):
        spec = LayerSpec("ep", M, K, N, r, act="outlier", outlier_frac=0.01, outlier_mult=20.0, seed=seed, bias=bias,
                         group=group)
        self.spec, self.cpu = spec, make_layer(spec)
        d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        lay = self.cpu
        self.X = d(lay.X)
        if r == 0:
            lay.L1 = lay.L2 = None
        self.fmt = fmt
        if fmt == "nvfp4":
            self.pl = hsq.Fp4Linear(d(lay.W), d(lay.s), d(lay.L1), d(lay.L2), d(lay.bias))
        else:
            self.pl = hsq.PackedLinear(d(lay.W), d(lay.s), d(lay.L1), d(lay.L2), d(lay.bias), group=group)

    def __call__(self, form, Y, epilogue=None):
        M, out = Y.shape[0], hsq.HSQ_OUT_F32 if Y.dtype == torch.float32 else hsq.HSQ_OUT_BF16
        s = self.spec
        if self.fmt == "nvfp4":
            act = hsq.Fp4ActBuffers(M, s.K, s.r, DEV)
            return hsq.fp4_forward(self.pl, self.X, act, Y, out=out, epilogue=epilogue)
        if form == "fused":
            return hsq.forward_fused(self.pl, self.X, Y, out=out, epilogue=epilogue)
        if form == "x":
            return hsq.forward_x(self.pl, self.X, Y, self.pl.workspace_x(M), out=out, epilogue=epilogue)
        act = hsq.ActBuffers(M, s.K, s.r, DEV, s.group)
        return hsq.forward(self.pl, self.X, act, Y, workspace=self.pl.workspace(M), out=out, epilogue=epilogue)


# (form, fmt, M, K, N, r, group): every kernel family, odd sizes, several tiles, split sums
SHAPES = [
    ("codes", "int4", 1, 192, 264, 4, 64),       # weight stream
    ("codes", "int4", 7, 1152, 136, 0, 128),     # ... 8-token kernel, two of them
    ("fused", "int4", 1, 1024, 520, 4, 64),      # single launch, stream form
    ("fused", "int4", 4, 512, 264, 2, 128),
    ("fused", "int4", 3, 640, 8, 1, 64),
    ("fused", "int4", 5, 1152, 520, 4, 64),      # single launch, decode tiles
    ("fused", "int4", 16, 4096, 264, 32, 128),   # ... split sums
    ("codes", "int4", 13, 2048, 392, 5, 64),     # decode tiles, 16 tokens, split sums
    ("codes", "int4", 29, 576, 1160, 4, 128),
    ("x", "int4", 32, 2048, 128, 4, 64),
    ("codes", "int4", 63, 1152, 392, 16, 64),
    ("x", "int4", 48, 640, 520, 0, 128),
    ("codes", "int4", 100, 1152, 776, 4, 64),    # mid tiles
    ("x", "int4", 250, 512, 264, 32, 64),
    ("codes", "int4", 129, 384, 520, 4, 128),    # large tiles, groups of 128
    ("x", "int4", 700, 1152, 1160, 4, 64),
    ("codes", "int4", 300, 896, 264, 20, 128),
    ("x", "int4", 3700, 256, 520, 4, 64),        # activations written as expanded tiles
    ("codes", "nvfp4", 1, 192, 264, 4, 64),
    ("codes", "nvfp4", 130, 320, 392, 0, 64),
    ("codes", "nvfp4", 1000, 512, 2056, 32, 64),
    ("x", "int4", 520, 640, 392, 32, 64),        # large tiles, many ranks
]
ACTS = ["silu", "gelu_tanh", "gelu_erf", "relu", "none"]


@pytest.mark.parametrize("i", range(len(SHAPES)), ids=lambda i: "-".join(map(str, SHAPES[i])))
def test_epilogue_against_fp64(i):
    form, fmt, M, K, N, r, group = SHAPES[i]
    lay = Layer(M, K, N, r, group, fmt, seed=i, bias=i % 2 == 0)
    z = torch.empty(M, N, device=DEV)
    lay(form, z)
    g = torch.Generator(device=DEV).manual_seed(i)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    full = rnd(M, 2 * N).to(torch.bfloat16)[:, N:]                 # a column range
    rows = max(1, -(-M // 3))
    sample = rnd(-(-M // rows), N)
    res32, res16 = rnd(M, N), rnd(M, N + 8).to(torch.bfloat16)[:, :N]
    for k, act in enumerate(ACTS):
        for out, mul, mr, res in ((torch.bfloat16, full, 1, None), (torch.float32, sample, rows, res16),
                                  (torch.bfloat16, None, 1, res32), (torch.float32, full, 1, res32),
                                  (torch.bfloat16, None, 1, None)):
            buf = torch.full((M + 2, N), 7.5, device=DEV, dtype=out)  # rows in front of and behind Y
            Y = buf[1:M + 1]
            if Y.data_ptr() % 16:
                pytest.fail("sentinel row breaks the alignment")
            lay(form, Y, hsq.Epilogue(act, mul=mul, mul_rows=mr, residual=res))
            y, tol = _expect(z, act, mul, mr, res)
            _check(Y, y, tol, f"{SHAPES[i]} {act} {out} mul {mr if mul is not None else None} res {res is not None}")
            assert (buf[0] == 7.5).all() and (buf[-1] == 7.5).all()
    assert hsq.hsq_get_device_status() == hsq.HSQ_OK


@pytest.mark.parametrize("i", [0, 2, 6, 7, 12, 15, 20])
def test_empty_epilogue_is_the_plain_forward(i):
    form, fmt, M, K, N, r, group = SHAPES[i]
    lay = Layer(M, K, N, r, group, fmt, seed=i)
    for dt in (torch.bfloat16, torch.float32):
        a, b = (torch.empty(M, N, device=DEV, dtype=dt) for _ in range(2))
        lay(form, a)
        lay(form, b, hsq.Epilogue())
        assert torch.equal(a, b)


@pytest.mark.parametrize("i", [0, 2, 6, 7, 10, 12, 15, 17, 20])
def test_in_place_residual_and_mul(i):
    """Y as its own residual, and as its own multiplier, equal the call with copies, bit for bit."""
    form, fmt, M, K, N, r, group = SHAPES[i]
    lay = Layer(M, K, N, r, group, fmt, seed=i)
    for dt in (torch.bfloat16, torch.float32):
        old = torch.randn(M, N, device=DEV).to(dt)
        want = torch.empty_like(old)
        lay(form, want, hsq.Epilogue("silu", residual=old.clone()))
        Y = old.clone()
        lay(form, Y, hsq.Epilogue("silu", residual=Y))
        assert torch.equal(Y, want)
        lay(form, want, hsq.Epilogue("gelu_tanh", mul=old.clone(), residual=old.clone()))
        Y = old.clone()
        lay(form, Y, hsq.Epilogue("gelu_tanh", mul=Y, residual=Y))
        assert torch.equal(Y, want)


@pytest.mark.parametrize("M,K,group", [(3, 512, 64), (12, 2048, 64), (100, 640, 64), (300, 512, 128)])
def test_forward_without_allocation(M, K, group):
    """hsq_linear_forward_noalloc_ep, twice in a row: the bits of the call with a workspace."""
    lay = Layer(M, K, 392, 4, group, seed=M)
    pl, s = lay.pl, lay.spec
    res = torch.randn(M, 392, device=DEV).to(torch.bfloat16)
    ep = hsq.Epilogue("gelu_tanh", residual=res)
    want = torch.empty(M, 392, device=DEV, dtype=torch.bfloat16)
    lay("codes", want, ep)
    act = hsq.ActBuffers(M, K, 4, DEV, group)
    hsq.hsq_quantize_act(lay.X, pl.s, pl.L1, M, K, 4, act.x_codes, act.x_scales, act.U, group=group)
    for _ in range(2):
        Y = torch.empty_like(want)
        hsq.hsq_linear_forward_noalloc_ep(act.x_codes, act.x_scales, act.U, pl.w_codes, pl.w_scales, pl.L2, pl.bias, M,
                                          s.N, K, 4, Y, ep, group=group)
        assert torch.equal(Y, want)


@pytest.mark.parametrize("form,M", [("fused", 2), ("codes", 12), ("x", 150), ("x", 600)])
def test_large_values_and_non_finite_operands(form, M):
    """z far outside the exponential's range (through the bias), and infinities and NaN in mul and residual."""
    K, N = 256, 136
    lay = Layer(M, K, N, 4, seed=3)
    big = torch.tensor([-3e38, -1e30, -1e13, -1e4, -100.0, -88.0, -20.0, 0.0, 20.0, 88.0, 100.0, 1e4, 1e13, 1e30, 3e38],
                       device=DEV).to(torch.bfloat16)
    lay.pl.bias[:15] = big
    lay.pl.bias[120:135] = big
    z = torch.empty(M, N, device=DEV)
    lay(form, z)
    for act in ACTS:
        Y = torch.empty(M, N, device=DEV)
        lay(form, Y, hsq.Epilogue(act))
        if act == "none":
            assert torch.equal(Y, z)
            continue
        y, tol = _expect(z, act, None, 1, None)
        d = (Y.double() - y).abs()
        assert (d <= tol + y.abs() * U + 1e-35).all(), (act, float((d - tol).max()))
    res = torch.randn(M, N, device=DEV)
    res[0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1.0], device=DEV)
    mul = torch.ones(M, N, device=DEV, dtype=torch.bfloat16)
    mul[-1, 4:6] = torch.tensor([float("inf"), float("nan")], device=DEV, dtype=torch.bfloat16)
    Y = torch.empty(M, N, device=DEV)
    lay.pl.bias.fill_(1.0)
    lay(form, Y, hsq.Epilogue("none", mul=mul, residual=res))
    assert Y[0, 0] == float("inf") and Y[0, 1] == -float("inf") and Y[0, 2].isnan()
    assert Y[-1, 4].isinf() and Y[-1, 5].isnan()
    ok = torch.ones_like(Y, dtype=torch.bool)
    ok[0, :3] = False
    ok[-1, 4:6] = False
    assert torch.isfinite(Y[ok]).all()


def test_epilogue_refusals_of_the_binding():
    lay = Layer(16, 64, 64, 4)
    Y = torch.empty(16, 64, device=DEV, dtype=torch.bfloat16)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, device=DEV, dtype=dt)  # noqa: E731
    for kw in (dict(mul=z(15, 64)), dict(mul=z(2, 64), mul_rows=7), dict(mul=z(16, 64), mul_rows=0),
               dict(residual=z(16, 72)), dict(residual=z(1, 64))):
        with pytest.raises(ValueError):
            lay("x", Y, hsq.Epilogue(**kw))
    for bad in (z(15, 64), z(16, 72), z(16, 64, dt=torch.float32), z(16, 64, dt=torch.float16)):  # not what is written
        with pytest.raises(ValueError):
            hsq.hsq_linear_forward_x_ep(lay.X, lay.pl.s, lay.pl.L1, lay.pl.w_codes, lay.pl.w_scales, None, lay.pl.L2,
                                        lay.pl.bias, 16, 64, 64, 4, bad, hsq.Epilogue("relu"),
                                        workspace=lay.pl.workspace_x(16), ws_bytes=lay.pl.workspace_x(16).numel())
    for kw in (dict(mul=z(64, 16).t()), dict(residual=z(16, 64, dt=torch.float16)), dict(residual=z(64))):
        with pytest.raises(ValueError):
            hsq.Epilogue(**kw)
    for kw, st in ((dict(residual=z(16, 65)[:, :64]), hsq.HSQ_ERR_UNSUPPORTED),
                   (dict(residual=z(16, 80)[:, 4:68]), hsq.HSQ_ERR_ALIGNMENT)):
        with pytest.raises(hsq.HsqError) as e:
            lay("x", Y, hsq.Epilogue(**kw))
        assert e.value.status == st
    wide = z(16, 128)
    with pytest.raises(hsq.HsqError):  # a Y inside the residual's rows
        hsq.hsq_linear_forward_x_ep(lay.X, lay.pl.s, lay.pl.L1, lay.pl.w_codes, lay.pl.w_scales, None, lay.pl.L2,
                                    lay.pl.bias, 16, 64, 64, 4, wide.view(-1)[:1024].view(16, 64),
                                    hsq.Epilogue(residual=wide[:, 64:]), workspace=lay.pl.workspace_x(16),
                                    ws_bytes=lay.pl.workspace_x(16).numel())
    assert hsq.hsq_get_device_status() == hsq.HSQ_OK


@pytest.mark.parametrize("form,M", [("fused", 1), ("fused", 9), ("x", 200), ("x", 1100)])
def test_captured_and_replayed_on_another_stream(form, M):
    """A captured gated MLP step, replayed with new inputs, equals eager calls."""
    K, N = 512, 520
    lay = Layer(M, K, N, 4, seed=M)
    mul = torch.randn(M, N, device=DEV).to(torch.bfloat16)
    res = torch.randn(M, N, device=DEV)
    Y, want = torch.empty(M, N, device=DEV), torch.empty(M, N, device=DEV)
    ws = lay.pl.workspace_x(M)
    ep = hsq.Epilogue("silu", mul=mul, residual=res)
    step = ((lambda out: hsq.forward_fused(lay.pl, lay.X, out, out=hsq.HSQ_OUT_F32, epilogue=ep)) if form == "fused" else
            (lambda out: hsq.forward_x(lay.pl, lay.X, out, ws, out=hsq.HSQ_OUT_F32, epilogue=ep)))
    step(Y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(Y)
    for k in range(3):
        mul.copy_(torch.randn(M, N, device=DEV))
        res.copy_(torch.randn(M, N, device=DEV))
        lay.X.copy_(torch.randn(M, K, device=DEV))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            g.replay()
        torch.cuda.current_stream().wait_stream(side)
        step(want)
        assert torch.equal(Y, want)
    torch.cuda.synchronize()


def test_offsets_pass_32_bits():
    """Y, mul and residual of more than 2^31 elements: the last rows equal a call on them alone (the same kernels: both
    are many tokens)."""
    M, K, N = 262144, 64, 8320
    lay = Layer(5000, K, N, 4, seed=1)
    X = torch.randn(M, K, device=DEV).to(torch.bfloat16)
    mul = torch.empty(M, N, device=DEV, dtype=torch.bfloat16)
    mul[-5000:] = torch.randn(5000, N, device=DEV)
    Y = torch.empty(M, N, device=DEV, dtype=torch.bfloat16)
    Y[-5000:] = torch.randn(5000, N, device=DEV)
    want, old = torch.empty(5000, N, device=DEV, dtype=torch.bfloat16), Y[-5000:].clone()
    hsq.forward_x(lay.pl, X, Y, lay.pl.workspace_x(M), epilogue=hsq.Epilogue("silu", mul=mul, residual=Y))
    hsq.forward_x(lay.pl, X[-5000:].clone(), want, lay.pl.workspace_x(5000),
                  epilogue=hsq.Epilogue("silu", mul=mul[-5000:], residual=old))
    assert torch.equal(Y[-5000:], want)
    assert hsq.hsq_get_device_status() == hsq.HSQ_OK


def test_epilogue_against_the_oracle():
    """The whole layer from the oracle's z in fp64: the spec's tolerance through the activation (|act'| <= 1.13)."""
    M, K, N, r = 37, 448, 264, 4
    lay = Layer(M, K, N, r, seed=9)
    c = lay.cpu
    z = torch.from_numpy(oracle_layer(c.X, c.W, c.s, c.L1, c.L2, c.bias)["Y"])
    mul, res = torch.randn(M, N), torch.randn(M, N)
    for act in ACTS:
        Y = torch.empty(M, N, device=DEV)
        lay("x", Y, hsq.Epilogue(act, mul=mul.to(DEV), residual=res.to(DEV)))
        y, tol = _expect(z, act, mul, 1, res)
        d = (Y.cpu().double() - y).abs()
        assert (d <= 1.13 * 1e-4 * rms(z.numpy()) * mul.abs().double() + tol + y.abs() * U).all(), act
