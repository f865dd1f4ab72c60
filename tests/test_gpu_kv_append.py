"""hsq_kv_append on the GPU against indexing in Python and rotation in fp64.

Tolerance of rotated values: as in test_gpu_rope (one rounding to the stored type).
E4M3: the stored byte is the nearest to x / scale, which the kernel has to 2^-22 of
scale-free |a| + |b| (the rotation) and 2^-24 (the quotient): half a step of the
byte's value (2^-4 relative, 2^-10 below the smallest normal) and that."""
import pytest
import torch

from test_gpu_rope import rotate64
from w4a4_rank_assisted_b200 import hsq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SMALL = 2.0 ** -22 + 2.0 ** -23


class Batch:
    """A packed batch: new tokens n_new[b] behind lens[b] cached ones, its pages scattered over a pool."""

    def __init__(self, n_new, lens, page, kv, q, D, dtype, cache, layout="slots", pad=0, cu=True, seed=0, spare=3,
                 first=0):
        g = torch.Generator().manual_seed(seed)
        self.n_new, self.lens, self.page = n_new, lens, page
        B, real = len(n_new), sum(n_new)
        T = first + real + pad
        self.first, self.T, self.real = first, T, real
        need = [-(-max(0, a + n) // page) if a >= 0 else 1 for a, n in zip(lens, n_new)]
        cols = max(max(need), 1) + 1
        pages = sum(need) + spare
        perm = torch.randperm(pages, generator=g).tolist()
        table = torch.full((B, cols), -1, dtype=torch.int32)
        for b, k in enumerate(need):
            for j in range(k):
                table[b, j] = perm.pop()
        self.table = table.to(DEV)
        qkv = torch.randn(T, q + 2 * kv, D, generator=g).to(dtype).to(DEV)
        self.qkv, self.q, self.k, self.v = qkv, qkv[:, :q], qkv[:, q:q + kv], qkv[:, q + kv:]
        shape = (pages, page, kv, D) if layout != "heads" else (pages, kv, page, D)
        mk = lambda: (torch.randn(shape, generator=g) * 3).to(cache).to(DEV)  # noqa: E731
        self.kc, self.vc = mk(), mk()
        if layout == "heads":
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        if layout == "pool":  # k and v as the two halves of every page
            both = torch.stack((self.kc, self.vc), 1).contiguous()
            self.kc, self.vc = both[:, 0], both[:, 1]
        self.q_out = torch.full((T, q, D), 9.0, device=DEV, dtype=dtype) if q else None
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
        c = [first]
        for n in n_new:
            c.append(c[-1] + n)
        self.cu = torch.tensor(c, dtype=torch.int32, device=DEV) if cu else None

    def places(self):
        """(token, sequence, place) of the tokens that take part."""
        t = self.first
        for b, n in enumerate(self.n_new):
            for i in range(n):
                if self.lens[b] >= 0:
                    yield t, b, self.lens[b] + i
                t += 1


def run_and_check(b, rotation=None, freqs=None, adjacent=False, positions=None, axes=None, k_scale=None, v_scale=None,
                  q_in_place=False):
    kc0, vc0 = b.kc.float().cpu(), b.vc.float().cpu()
    q0, k0, v0 = b.qkv.clone()[:, :b.q.shape[1]], b.k.clone(), b.v.clone()
    has_q = b.q.shape[1] > 0
    q_out = b.q if q_in_place else b.q_out
    before = None if not has_q else q_out.clone()
    hsq.hsq_kv_append(b.k, b.v, b.kc, b.vc, b.table, b.lens_t, cu_seqlens=b.cu, rotation=rotation, positions=positions,
                      q=b.q if has_q else None, q_out=q_out if has_q else None, k_scale=k_scale, v_scale=v_scale)
    assert hsq.hsq_get_device_status() == hsq.HSQ_OK
    places = list(b.places())
    D = b.k.shape[2]
    tok = torch.tensor([t for t, _, _ in places], dtype=torch.long)
    at = torch.tensor([p for _, _, p in places], dtype=torch.float64)
    sc = 1.0 if rotation is None else rotation.scale
    if rotation is not None:
        p = at[:, None] if positions is None else positions.cpu().double().view(b.T, -1)[tok]
        ax = torch.tensor(axes if axes is not None else [0] * len(freqs))
        ang = (p[:, ax] if positions is not None else p) * freqs.cpu().double()
    turn = lambda x: (rotate64(x.cpu()[tok], ang, adjacent, scale=sc) if rotation is not None  # noqa: E731
                      else (x.cpu()[tok].double(), torch.zeros(len(tok), x.shape[1], D, dtype=torch.float64)))
    kw, km = turn(k0)
    vw, vm = v0.cpu()[tok].double(), torch.zeros(len(tok), v0.shape[1], D, dtype=torch.float64)
    table = b.table.cpu()
    touched = torch.zeros(b.kc.shape[:2], dtype=torch.bool)
    for name, cache, old, want, m, scale in (("k", b.kc, kc0, kw, km, k_scale), ("v", b.vc, vc0, vw, vm, v_scale)):
        got = cache.float().cpu().double()
        exp, tol = old.double().clone(), torch.zeros_like(got)
        for i, (t, s, p) in enumerate(places):
            page, slot = int(table[s, p // b.page]), p % b.page
            touched[page, slot] = True
            w, e = want[i], m[i] * SMALL
            if cache.dtype == torch.float8_e4m3fn:
                if scale is not None:
                    w, e = w / scale.cpu().double()[:, None], e / scale.cpu().double()[:, None]
                e = e + w.abs() * 2.0 ** -24
                w = w.clamp(-448, 448)
                e = e + torch.maximum((w.abs() + e) * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
            else:
                half = 2.0 ** -8 if cache.dtype == torch.bfloat16 else 2.0 ** -24
                e = e * (1 + half) + w.abs() * half * (1.0 if (m[i] > 0).any() or b.k.dtype != cache.dtype else 0.0)
            exp[page, slot], tol[page, slot] = w, e
        d = (got - exp).abs()
        assert (d <= tol).all(), f"{name}: worst {float((d - tol).max()):.3e} over"
        assert torch.equal(got[~touched], old.double()[~touched])
    if has_q:
        qw, qm = turn(q0)
        got = q_out.cpu().double()
        half = 2.0 ** -8 if b.k.dtype == torch.bfloat16 else 2.0 ** -24
        assert ((got[tok] - qw).abs() <= qm * SMALL * (1 + half) + qw.abs() * half).all()
        rest = torch.ones(b.T, dtype=torch.bool)
        rest[tok] = False
        assert torch.equal(q_out.cpu()[rest], before.cpu()[rest])
    assert torch.equal(b.k, k0) and torch.equal(b.v, v0)


def ladder(P):
    return (10000.0 ** (-torch.arange(P, dtype=torch.float64) / P)).float().to(DEV)


BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
# (n_new, lens, page, kv, q, D, dtype, cache, layout, pad, pairs, adjacent)
CASES = [
    ([1], [0], 16, 8, 32, 128, BF, BF, "slots", 0, 64, False),           # the first token of all
    ([1], [70000], 16, 1, 4, 128, BF, BF, "slots", 0, 64, False),        # far along
    ([5], [0], 1, 2, 6, 64, BF, BF, "slots", 0, 32, True),               # pages of one token
    ([0, 3, 0, 20, 1, 0], [5, 15, 3, 16, 31, 0], 16, 2, 8, 64, BF, F8, "slots", 4, 32, False),
    ([9, 30, 2], [7, 0, 23], 24, 3, 3, 80, BF, BF, "heads", 1, 40, False),  # 24 tokens a page, ends inside pages
    ([9, 30, 2], [7, 0, 23], 24, 3, 3, 80, F32, BF, "heads", 1, 40, False),
    ([17, 1], [100, 3], 32, 4, 0, 72, BF, BF, "slots", 0, 36, False),    # 8-byte pieces, no queries
    ([17, 1], [100, 3], 32, 4, 4, 72, F32, F8, "slots", 0, 36, True),
    ([17, 1], [100, 3], 32, 4, 4, 72, BF, F32, "pool", 0, 36, False),
    ([4, 4], [1, 2], 8, 2, 2, 50, BF, BF, "slots", 3, 25, False),        # single elements
    ([4, 4], [1, 2], 8, 2, 2, 7, F32, F8, "slots", 0, 2, True),          # odd head, three elements pass
    ([4, 6], [1, 2], 8, 2, 4, 128, BF, F32, "pool", 0, 32, False),
    ([40, 6], [1, 200], 128, 8, 56, 128, BF, BF, "slots", 0, 64, True),
    ([300, 1, 513], [77, 999, 0], 64, 8, 32, 128, BF, BF, "heads", 9, 64, False),
    ([3, 5], [-1, 6], 8, 2, 4, 64, BF, BF, "slots", 0, 32, False),       # a sequence that takes no part
    ([6], [3], 4, 2, 4, 512, F32, F32, "slots", 0, 256, False),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_append_against_indexing(i):
    n_new, lens, page, kv, q, D, dtype, cache, layout, pad, P, adjacent = CASES[i]
    f = ladder(P)
    scale = [0.02 + 0.1 * torch.rand(kv, device=DEV) for _ in range(2)] if cache == F8 else [None, None]
    for rot in (hsq.Rotation(f, interleaved=adjacent), None):
        b = Batch(n_new, lens, page, kv, q, D, dtype, cache, layout, pad, seed=i, first=i % 3)
        run_and_check(b, rot, f, adjacent, k_scale=scale[0], v_scale=scale[1])
    b = Batch(n_new, lens, page, kv, q, D, dtype, cache, layout, pad, seed=i)
    rot = hsq.Rotation(f, interleaved=adjacent, scale=0.5)
    run_and_check(b, rot, f, adjacent, k_scale=scale[0], q_in_place=True)


@pytest.mark.parametrize("cache", [BF, F8], ids=["bf16", "e4m3"])
def test_decode_batch(cache):
    """One token per sequence, without cu_seqlens; one sequence inactive."""
    lens = [0, 15, 16, 17, 4000, -1, 31, 32, 1, 255]
    b = Batch([1] * 10, lens, 16, 8, 32, 128, BF, cache, cu=False)
    f = ladder(64)
    run_and_check(b, hsq.Rotation(f), f)


def test_positions_of_their_own():
    """Three axes whose positions are not the cache's places (an image inside a prompt)."""
    b = Batch([9, 14], [3, 40], 16, 2, 6, 128, BF, BF, pad=2)
    f = ladder(64)
    axes = [0] * 16 + [1] * 24 + [2] * 24
    for pos in (torch.randint(0, 900, (b.T, 3), device=DEV, dtype=torch.int32),
                torch.rand(b.T, 3, device=DEV) * 100):
        run_and_check(b, hsq.Rotation(f, axes), f, positions=pos, axes=axes)


def test_e4m3_saturates_and_keeps_nan():
    b = Batch([4], [0], 4, 1, 0, 16, BF, F8)
    b.v[0, 0, :6] = torch.tensor([1e30, -1e30, float("inf"), -float("inf"), float("nan"), 0.0], device=DEV)
    b.v[1, 0, :4] = torch.tensor([448.0, 464.0, 2.0 ** -9, 2.0 ** -10], device=DEV)  # 464 and 2^-10 are ties
    hsq.hsq_kv_append(b.k, b.v, b.kc, b.vc, b.table, b.lens_t, cu_seqlens=b.cu)
    page = int(b.table[0, 0])
    got = b.vc[page].float()
    assert got[0, 0, :4].tolist() == [448.0, -448.0, 448.0, -448.0] and got[0, 0, 4].isnan() and got[0, 0, 5] == 0
    assert got[1, 0, :4].tolist() == [448.0, 448.0, 2.0 ** -9, 0.0]


def test_values_are_copied_whatever_they_are():
    """Without a change of type v is a copy, bit for bit; a NaN in k stays in its pair."""
    b = Batch([5], [2], 4, 2, 2, 64, BF, BF)
    b.v[0, 0, :3] = torch.tensor([float("nan"), float("inf"), -0.0], device=DEV)
    b.k[1, 1, 3] = float("nan")
    f = ladder(32)
    hsq.hsq_kv_append(b.k, b.v, b.kc, b.vc, b.table, b.lens_t, cu_seqlens=b.cu, rotation=hsq.Rotation(f))
    for t, s, p in b.places():
        page, slot = int(b.table[s, p // 4]), p % 4
        assert torch.equal(b.vc[page, slot].view(torch.int16), b.v[t].view(torch.int16))
        nan = b.kc[page, slot].isnan()
        want = torch.zeros_like(nan)
        if t == 1:
            want[1, 3] = want[1, 35] = True
        assert torch.equal(nan, want)


def test_bad_pages_are_reported_and_not_written():
    """Page numbers outside the cache and places behind the table: those tokens' k and v are skipped, the rest of
    the call is done, and the status says so once."""
    f = ladder(64)
    for what in ("negative", "large", "behind"):
        b = Batch([4, 4, 4], [0, 6, 0], 8, 2, 4, 128, BF, BF, seed=5)
        table = b.table
        if what == "negative":
            table[0, 0] = -1
        elif what == "large":
            table[0, 0] = b.kc.shape[0]
        else:
            table = table[:, :1].contiguous()  # sequence 1 needs a second page
        kc0, vc0 = b.kc.clone(), b.vc.clone()
        hsq.hsq_kv_append(b.k, b.v, b.kc, b.vc, table, b.lens_t, cu_seqlens=b.cu, rotation=hsq.Rotation(f), q=b.q,
                          q_out=b.q_out)
        assert hsq.hsq_get_device_status() == hsq.HSQ_ERR_BAD_PAGE
        assert hsq.hsq_get_device_status() == hsq.HSQ_OK
        touched = torch.zeros(b.kc.shape[:2], dtype=torch.bool, device=DEV)
        for t, s, p in b.places():
            if (what == "behind" and p >= 8) or (what != "behind" and s == 0):
                continue
            page, slot = int(b.table[s, p // 8]), p % 8
            touched[page, slot] = True
            assert torch.equal(b.vc[page, slot], b.v[t])
        assert torch.equal(b.kc[~touched], kc0[~touched]) and torch.equal(b.vc[~touched], vc0[~touched])
        assert (b.q_out != 9.0).any(-1).all()  # the queries are rotated all the same


def test_graph_replay_with_changed_lengths():
    """A captured decode step: lens, table and inputs change between replays."""
    f = ladder(64)
    rot = hsq.Rotation(f)
    b = Batch([1] * 6, [3, 7, 15, 16, 0, 30], 16, 4, 8, 128, BF, BF, cu=False, spare=20)
    b.table[b.table < 0] = 0  # the graph's later steps reach the next column
    kc, vc, qo = b.kc.clone(), b.vc.clone(), b.q_out.clone()
    call = lambda kc, vc, qo: hsq.hsq_kv_append(b.k, b.v, kc, vc, b.table, b.lens_t, rotation=rot, q=b.q, q_out=qo)  # noqa: E731
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        call(b.kc, b.vc, b.q_out)
    used = set(b.table[:, 0].tolist()) | set(b.table[:, 1].tolist())
    free = [p for p in range(b.kc.shape[0]) if p not in used]
    for c in range(6):  # a page of its own for every next column
        b.table[c, 1] = free.pop() if c != 3 and c != 5 else b.table[c, 1]
        b.table[c, 2:] = free[0]
    for k in range(3):
        b.qkv.copy_(torch.randn(b.qkv.shape, device=DEV))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            g.replay()
        torch.cuda.current_stream().wait_stream(side)
        call(kc, vc, qo)
        assert torch.equal(b.kc, kc) and torch.equal(b.vc, vc) and torch.equal(b.q_out, qo)
        b.lens_t += 1
    torch.cuda.synchronize()


def test_two_appends_at_once():
    """Two batches into caches of their own, on two streams: each as alone."""
    f = ladder(64)
    rot = hsq.Rotation(f)
    b = [Batch([200, 40, 7], [3, 60, 0], 16, 4, 8, 128, BF, BF, seed=s, cu=True) for s in (1, 2)]
    alone = []
    for x in b:
        kc, vc, q = x.kc.clone(), x.vc.clone(), x.q_out.clone()
        hsq.hsq_kv_append(x.k, x.v, kc, vc, x.table, x.lens_t, cu_seqlens=x.cu, rotation=rot, q=x.q, q_out=q)
        alone.append((kc, vc, q))
    streams = [torch.cuda.Stream() for _ in b]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, st in zip(b, streams):
            hsq.hsq_kv_append(x.k, x.v, x.kc, x.vc, x.table, x.lens_t, cu_seqlens=x.cu, rotation=rot, q=x.q, q_out=x.q_out,
                              stream=st)
    torch.cuda.synchronize()
    for x, want in zip(b, alone):
        assert all(torch.equal(g, w) for g, w in zip((x.kc, x.vc, x.q_out), want))


def test_long_cache_offsets_pass_32_bits():
    """A cache of more than 2^31 elements: its last pages are reached (bf16, 4.6 GB each of k and v)."""
    page, kv, D = 64, 8, 128
    pages = (1 << 31) // (page * kv * D) + 2000
    kc = torch.zeros(pages, page, kv, D, device=DEV, dtype=BF)
    vc = torch.zeros_like(kc)
    k, v = torch.randn(2, kv, D, device=DEV).to(BF), torch.randn(2, kv, D, device=DEV).to(BF)
    table = torch.tensor([[pages - 1], [0]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([63, 0], dtype=torch.int32, device=DEV)
    hsq.hsq_kv_append(k, v, kc, vc, table, lens)
    assert torch.equal(kc[pages - 1, 63], k[0]) and torch.equal(vc[pages - 1, 63], v[0])
    assert torch.equal(kc[0, 0], k[1]) and not kc[0, 1:].any() and not kc[1:pages - 1].any()
    assert hsq.hsq_get_device_status() == hsq.HSQ_OK


def test_refusals_of_the_binding():
    b = Batch([2, 1], [3, 4], 8, 2, 4, 64, BF, BF)
    base = dict(k=b.k, v=b.v, k_cache=b.kc, v_cache=b.vc, block_table=b.table, cache_lens=b.lens_t, cu_seqlens=b.cu)
    bad = [dict(v=b.v.float()), dict(k=b.k.half(), v=b.v.half()), dict(v=b.v[:, :1]), dict(k_cache=b.kc[:, :4]),
           dict(k_cache=b.kc.half(), v_cache=b.vc.half()), dict(v_cache=b.vc.transpose(1, 2).contiguous().transpose(1, 2)),
           dict(block_table=b.table.long()), dict(cache_lens=b.lens_t[:1]), dict(cu_seqlens=b.cu[:2]),
           dict(q=b.q), dict(q=b.q[:2], q_out=b.q_out[:2]), dict(q=b.q, q_out=b.q_out.float()),
           dict(k_scale=torch.ones(3, device=DEV)), dict(positions=torch.arange(3, device=DEV)),
           dict(block_table=b.table.cpu())]
    for kw in bad:
        with pytest.raises(ValueError):
            hsq.hsq_kv_append(**{**base, **kw})
    for kw in (dict(k_scale=torch.ones(2, device=DEV)),                     # scales for a bf16 cache
               dict(cu_seqlens=None),                                       # 3 tokens, 2 sequences
               dict(v_cache=b.kc),                                          # one cache for both
               dict(q=b.q, q_out=b.qkv[:, 2:6])):                           # q_out over k
        with pytest.raises(hsq.HsqError):
            hsq.hsq_kv_append(**{**base, **kw})
    hsq.hsq_kv_append(**{**base, "k": b.k[:0], "v": b.v[:0]})  # no new tokens: nothing to do
    assert hsq.hsq_get_device_status() == hsq.HSQ_OK
