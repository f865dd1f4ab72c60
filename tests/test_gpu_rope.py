"""hsq_rope on the GPU against the rotation in fp64.

Tolerance: the angle's remainder, rounded to fp32 turns below 1/2, is off by at most
2^-25 * 2 pi and its sine and cosine by 2 ulp more (2^-22 of 1); each output is two
products and a sum of those: |y| off by (2^-22 + 2^-23) scale (|a| + |b|) before it
is rounded (half a step: 2^-24 relative for fp32, 2^-8 for bf16)."""
import pytest
import torch

from w4a4_rank_assisted_b200 import hsq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def angles(pos, freqs, axes):
    """[rows, pairs] in fp64, on the CPU."""
    p = pos.cpu().double()
    p = p[:, None] if p.dim() == 1 else p
    return p[:, axes] * freqs.cpu().double()


def rotate64(x, ang, adjacent, transpose=False, scale=1.0):
    """(rotation of x [T, H, D] in fp64, scale * (|a| + |b|) of every element), by explicit 2 x 2 products."""
    x = x.cpu().double()
    P = ang.shape[1]
    i = torch.arange(P)
    ia, ib = (2 * i, 2 * i + 1) if adjacent else (i, P + i)
    c, s = torch.cos(ang)[:, None] * scale, torch.sin(ang)[:, None] * scale
    s = -s if transpose else s
    y, m = x.clone(), torch.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    m[..., ia] = m[..., ib] = abs(scale) * (a.abs() + b.abs())
    return y, m


def check(got, y, m, where=""):
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    d = (got.cpu().double() - y).abs()
    tol = m * (2.0 ** -22 + 2.0 ** -23) * (1 + half) + y.abs() * half * (m > 0)
    assert (d <= tol).all(), f"{where}: worst {float((d - tol).max()):.3e} over, at {int((d - tol).argmax())}"


# (tokens, heads, dim, pairs, axes, pos_rows)
CASES = [
    (1, 1, 2, 1, 1, 1),
    (1, 40, 128, 64, 1, 1),
    (3, 5, 128, 64, 3, 3),
    (7, 3, 72, 36, 2, 7),        # 8-byte pieces
    (33, 2, 80, 40, 4, 11),      # three samples that share their positions
    (5, 7, 128, 32, 3, 5),       # half of the head passes through
    (6, 3, 96, 20, 2, 6),        # ... its rest not a multiple of a piece
    (4, 2, 66, 33, 1, 2),        # single elements
    (9, 3, 7, 3, 2, 9),          # odd head
    (17, 6, 512, 256, 4, 17),
    (600, 9, 64, 32, 1, 600),
    (2111, 24, 128, 64, 3, 2111),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_rope_against_fp64(case, adjacent, dtype):
    T, H, D, P, A, R = case
    g = torch.Generator().manual_seed(T * 31 + D)
    freqs = (10000.0 ** (-torch.arange(P, dtype=torch.float64) / P)).float().to(DEV)
    axes = torch.randint(0, A, (P,), generator=g)
    axes[-1] = A - 1
    wide = torch.randn(T, H + 3, D, generator=g).to(dtype).to(DEV)
    x = wide[:, 1:H + 1]
    for pdt in (torch.int32, torch.int64, torch.float32):
        pos = torch.randint(0, 5000, (R, A), generator=g)
        pos = (pos.float() * 0.25 if pdt == torch.float32 else pos.to(pdt)).to(DEV)
        if A == 1 and pdt == torch.int32:
            pos = pos[:, 0]
        for transpose, scale in ((False, 1.0), (True, 1.25)):
            rot = hsq.Rotation(freqs, axes.tolist(), interleaved=adjacent, transpose=transpose, scale=scale)
            ang = angles(pos, freqs, axes)[torch.arange(T) % R]
            want, m = rotate64(x, ang, adjacent, transpose, scale)
            y = torch.full((T, H, D), float("nan"), device=DEV, dtype=dtype)
            hsq.hsq_rope(x, y, pos, rot)
            check(y, want, m, f"{case} {pdt}")
            if 2 * P < D:
                assert torch.equal(y[..., 2 * P:], x[..., 2 * P:])
            # in place, inside the wider tensor: the same bits, and the neighbours as they were
            w2 = wide.clone()
            hsq.hsq_rope(w2[:, 1:H + 1], w2[:, 1:H + 1], pos, rot)
            assert torch.equal(w2[:, 1:H + 1], y)
            assert torch.equal(w2[:, :1], wide[:, :1]) and torch.equal(w2[:, H + 1:], wide[:, H + 1:])


def _plain(T=5, H=4, D=64, P=32, dtype=torch.float32, seed=0):
    g = torch.Generator().manual_seed(seed)
    freqs = (10000.0 ** (-torch.arange(P, dtype=torch.float64) / P)).float().to(DEV)
    return torch.randn(T, H, D, generator=g).to(dtype).to(DEV), freqs


def test_far_positions():
    """Positions up to 10^8 with a frequency of 1, and negative ones: fp32 angles would be off by radians."""
    x, freqs = _plain(T=8)
    pos = torch.tensor([0, 1, -1, 99999, 10 ** 6, 2 ** 24 + 1, 10 ** 8, -(10 ** 8)], device=DEV)
    y = torch.empty_like(x)
    hsq.hsq_rope(x, y, pos, hsq.Rotation(freqs))
    # the fp64 angle itself (a product rounded at 2^-53) and its quotient by 2 pi: 10^8 * 2^-51 = 4e-8 more
    want, m = rotate64(x, angles(pos, freqs, torch.zeros(32, dtype=torch.long)), False)
    d = (y.cpu().double() - want).abs()
    assert (d <= m * (2.0 ** -22 + 2.0 ** -23 + 1e-7) + want.abs() * 2.0 ** -24).all()


@pytest.mark.parametrize("adjacent", [False, True])
def test_transpose_is_the_gradient(adjacent):
    """<rope(x), g> = <x, rope^T(g)>, and rope^T(g) against central differences of <rope(x), g> (the map is
    linear, so a difference of any step is exact up to the two rounded evaluations)."""
    x, freqs = _plain(T=6, H=3, D=80, P=32)
    g = _plain(T=6, H=3, D=80, P=32, seed=1)[0]
    pos = torch.randint(0, 300, (6, 3), device=DEV)
    axes = [i % 3 for i in range(32)]
    y, gx = torch.empty_like(x), torch.empty_like(x)
    fwd = hsq.Rotation(freqs, axes, interleaved=adjacent, scale=0.75)
    hsq.hsq_rope(x, y, pos, fwd)
    hsq.hsq_rope(g, gx, pos, hsq.Rotation(freqs, axes, interleaved=adjacent, scale=0.75, transpose=True))
    n = x.numel()
    a, b = (y.double() * g.double()).sum(), (x.double() * gx.double()).sum()
    # every element of both sums is off by at most (2^-22 + 2^-23 + 2^-24) * 2 max * max
    lim = n * 2 * 2.0 ** -21 * float(x.abs().max()) * float(g.abs().max())
    assert abs(float(a - b)) <= lim
    for at in ((0, 0, 0), (3, 1, 33), (5, 2, 63), (2, 0, 79)):
        up, dn, e = x.clone(), x.clone(), 2.0
        up[at] += e
        dn[at] -= e
        yu, yd = torch.empty_like(x), torch.empty_like(x)
        hsq.hsq_rope(up, yu, pos, fwd)
        hsq.hsq_rope(dn, yd, pos, fwd)
        num = float(((yu.double() - yd.double()) * g.double()).sum()) / (2 * e)
        lim = 80 * 2.0 ** -20 * float(g.abs().max()) * (float(x.abs().max()) + 2)
        assert abs(num - float(gx[at])) <= lim


def test_layouts_and_alignments():
    """Heads outside tokens, broadcast inputs, rows off 16 bytes: the values of the dense call."""
    T, H, D, P = 11, 3, 64, 32
    for dtype in (torch.bfloat16, torch.float32):
        x, freqs = _plain(T, H, D, P, dtype)
        pos = torch.arange(T, device=DEV, dtype=torch.int32) * 7
        rot = hsq.Rotation(freqs)
        want = torch.empty_like(x)
        hsq.hsq_rope(x, want, pos, rot)
        heads_first = x.transpose(0, 1).contiguous().transpose(0, 1)
        y = torch.empty(H, T, D, device=DEV, dtype=dtype).transpose(0, 1)
        hsq.hsq_rope(heads_first, y, pos, rot)
        assert torch.equal(y, want)
        flat = torch.zeros(T * H * D + 1, device=DEV, dtype=dtype)
        flat[1:] = x.flatten()
        off = flat[1:].view(T, H, D)
        y = torch.empty_like(x)
        hsq.hsq_rope(off, y, pos, rot)
        assert torch.equal(y, want)
        buf = torch.full((T, H, D + 1), 5.0, device=DEV, dtype=dtype)
        hsq.hsq_rope(x, buf[..., :D], pos, rot)
        assert torch.equal(buf[..., :D], want) and (buf[..., D] == 5).all()
        one = x[:, :1].expand(T, H, D)
        y = torch.empty_like(x)
        hsq.hsq_rope(one, y, pos, rot)
        assert torch.equal(y, want[:, :1].expand(T, H, D))
        wide_pos = torch.zeros(T, 4, device=DEV, dtype=torch.int32)
        wide_pos[:, 2] = pos
        hsq.hsq_rope(x, y, wide_pos[:, 2:3], rot)
        assert torch.equal(y, want)


def test_non_finite_values_stay_in_their_pair():
    x, freqs = _plain(T=3, H=2, D=64, P=16)
    x[1, 0, 5] = float("nan")
    x[1, 1, 40] = float("inf")  # behind the rotated part: passes through
    pos = torch.tensor([3, 4, 5], device=DEV)
    y = torch.empty_like(x)
    hsq.hsq_rope(x, y, pos, hsq.Rotation(freqs))
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 0, 5] = want[1, 0, 21] = want[1, 1, 40] = True
    assert torch.equal(bad, want) and y[1, 1, 40] == float("inf")


def test_offsets_pass_32_bits():
    """More than 2^31 elements of x and y: the last tokens equal a call on them alone."""
    T, H, D = 70000, 64, 512
    freqs = _plain()[1]
    x = torch.empty(T, H, D, device=DEV, dtype=torch.bfloat16)
    x[-3:] = torch.randn(3, H, D, device=DEV)
    x[:2] = torch.randn(2, H, D, device=DEV)
    pos = torch.arange(T, device=DEV)
    y, rot = torch.empty_like(x), hsq.Rotation(freqs, interleaved=True)
    hsq.hsq_rope(x, y, pos, rot)
    for part in (slice(0, 2), slice(T - 3, T)):
        want = torch.empty_like(x[part])
        hsq.hsq_rope(x[part], want, pos[part], rot)
        assert torch.equal(y[part], want)


def test_refusals_of_the_binding():
    x, freqs = _plain()
    rot, pos, y = hsq.Rotation(freqs), torch.arange(5, device=DEV), torch.empty_like(x)
    bad = [(x, y.to(torch.bfloat16), pos, rot), (x.half(), y.half(), pos, rot), (x, y[:, :3], pos, rot),
           (x, y, pos.to(torch.int16), rot), (x, y, pos[:, None].expand(5, 2).contiguous(), rot),
           (x[..., ::2], y[..., ::2], pos, rot), (x.cpu(), y.cpu(), pos, rot), (x, y, pos.cpu(), rot)]
    for a in bad:
        with pytest.raises(ValueError):
            hsq.hsq_rope(*a)
    for kw in (dict(freqs=freqs.double()), dict(freqs=freqs.cpu()), dict(freqs=freqs[::2]),
               dict(freqs=freqs, pair_axes=[0] * 31), dict(freqs=freqs, pair_axes=[4] * 32),
               dict(freqs=freqs, pair_axes=[-1] * 32)):
        with pytest.raises(ValueError):
            hsq.Rotation(**kw)
    with pytest.raises(hsq.HsqError):
        hsq.hsq_rope(x, y, torch.arange(6, device=DEV), rot)
    with pytest.raises(hsq.HsqError):
        hsq.hsq_rope(x, y, pos, hsq.Rotation(freqs, scale=0.0))
    two = torch.zeros(6, 4, 64, device=DEV)
    with pytest.raises(hsq.HsqError):
        hsq.hsq_rope(two[:5], two[1:], pos, rot)
    none = x[:0]
    hsq.hsq_rope(none, none, pos[:0], rot)  # nothing to do


def test_streams_and_graph():
    x, freqs = _plain(T=64, H=8, D=128, P=64, dtype=torch.bfloat16)
    pos = torch.arange(64, device=DEV)
    rot = hsq.Rotation(freqs)
    want, y = torch.empty_like(x), torch.zeros_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    hsq.hsq_rope(x, y, pos, rot, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    hsq.hsq_rope(x, want, pos, rot)
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hsq.hsq_rope(x, y, pos, rot)
    for k in range(2):
        pos += 13
        x.copy_(torch.randn(64, 8, 128, device=DEV))
        g.replay()
        hsq.hsq_rope(x, want, pos, rot)
        assert torch.equal(y, want)
