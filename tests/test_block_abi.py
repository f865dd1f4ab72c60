"""Host-side checks of the calls around a linear (no GPU needed): the epilogue,
the rotation and the cache append refuse what they do not take before anything is
launched, and calls of zero tokens do nothing."""
import ctypes

import pytest
import torch

from w4a4_rank_assisted_b200 import hsq

A = 1 << 20          # fake, non-null, 16-byte aligned device addresses, 1 MiB apart:
B = 2 << 20          # every call below must be refused before they are touched
C = 3 << 20
MIS = A + 4
INVALID, ALIGN, UNSUP = hsq.HSQ_ERR_INVALID_ARG, hsq.HSQ_ERR_ALIGNMENT, hsq.HSQ_ERR_UNSUPPORTED


def _epilogue(**kw):
    e = hsq._CEpilogue(act=4, mul_rows=1, mul_ld=64, residual_ld=64)
    for k, v in kw.items():
        setattr(e, k, v)
    return ctypes.byref(e)


def _forwards():
    """The calls with an epilogue on a 16 x 64 Y at address A (K = 64, r = 4)."""
    lib = hsq.load()
    far = 1 << 30
    return {
        "codes": lambda e: lib.hsq_linear_forward_ep(far, far, far, far, far, None, far, None, 16, 64, 64, 4, 64, A, 0, e,
                                                     far, 0, None),
        "noalloc": lambda e: lib.hsq_linear_forward_noalloc_ep(far, far, far, far, far, far, None, 16, 64, 64, 4, 64, A, 0,
                                                               e, None),
        "x": lambda e: lib.hsq_linear_forward_x_ep(far, far, far, far, far, None, far, None, 16, 64, 64, 4, 64, A, 0, e,
                                                   far, 0, None),
        "fused": lambda e: lib.hsq_linear_forward_fused_ep(far, far, far, far, far, far, None, 16, 64, 64, 4, 64, A, 0, e,
                                                           None),
        "fp4": lambda e: lib.hsq_fp4_linear_forward_ep(far, far, far, far, far, far, far, far, None, 16, 64, 64, 4, A, 0,
                                                       e, None),
    }


@pytest.mark.parametrize("form", ["codes", "noalloc", "x", "fused", "fp4"])
def test_epilogue_refusals(form):
    f = _forwards()[form]
    assert f(_epilogue(act=5)) == INVALID
    assert f(_epilogue(act=-1)) == INVALID
    assert f(_epilogue(mul=B, mul_dtype=2)) == INVALID
    assert f(_epilogue(mul=B, mul_rows=0)) == INVALID
    assert f(_epilogue(mul=B, mul_ld=56)) == INVALID            # narrower than N
    assert f(_epilogue(mul=B, mul_ld=68)) == UNSUP              # rows not on 8 elements
    assert f(_epilogue(mul=MIS + (1 << 22))) == ALIGN
    assert f(_epilogue(residual=B, residual_ld=0)) == INVALID
    assert f(_epilogue(residual=B, residual_dtype=7)) == INVALID
    assert f(_epilogue(residual=B + 8)) == ALIGN
    # operands that overlap Y (2048 bytes at A) without being it
    assert f(_epilogue(residual=A + 128)) == INVALID            # one row on
    assert f(_epilogue(residual=A, residual_dtype=1)) == INVALID  # the other type
    assert f(_epilogue(residual=A, residual_ld=128)) == INVALID
    assert f(_epilogue(mul=A, mul_rows=2)) == INVALID           # its rows are read by other tokens
    assert f(_epilogue(mul=A - 128, mul_rows=16, mul_ld=64, residual=A + 2048 - 16)) == INVALID


def test_fused_epilogue_refuses_y_over_x():
    lib = hsq.load()
    far = 1 << 30
    call = lambda X, Y: lib.hsq_linear_forward_fused_ep(X, far, far, far, far, far, None, 16, 64, 64, 4, 64, Y, 0,  # noqa: E731
                                                        _epilogue(), None)
    assert call(A, A) == INVALID and call(A, A + 1024) == INVALID


def test_epilogue_object_checks():
    with pytest.raises(ValueError):
        hsq.Epilogue("swish")
    with pytest.raises(ValueError):
        hsq.Epilogue("silu", mul=torch.zeros(4, 8))             # a CPU tensor


def _rope(x=(A, 512, 128), y=(B, 512, 128), dtype=0, tokens=3, heads=4, dim=128, rot=None, pos=None, no=()):
    r = dict(freqs=C, pair_axis=None, pairs=64, n_axes=1, interleaved=0, transpose=0, scale=1.0)
    r.update(rot or {})
    p = dict(data=C + 4096, type=0, rows=3, ld=1)
    p.update(pos or {})
    ref = ctypes.byref
    return hsq.load().hsq_rope(None if "x" in no else ref(hsq._CHeads(*x)), None if "y" in no else ref(hsq._CHeads(*y)),
                               dtype, tokens, heads, dim, None if "rot" in no else ref(hsq._CRotation(**r)),
                               None if "pos" in no else ref(hsq._CPositions(**p)), None)


def test_rope_refusals():
    for what in ("x", "y", "rot", "pos"):
        assert _rope(no=(what,)) == INVALID
    assert _rope(dtype=2) == INVALID                            # the cache's type is not a head's
    assert _rope(tokens=-1) == INVALID
    assert _rope(heads=0) == INVALID
    assert _rope(dim=1) == INVALID
    assert _rope(dim=514) == UNSUP
    assert _rope(rot=dict(freqs=None)) == INVALID
    assert _rope(rot=dict(pairs=0)) == INVALID
    assert _rope(rot=dict(pairs=65)) == INVALID
    assert _rope(rot=dict(n_axes=5)) == INVALID
    assert _rope(rot=dict(n_axes=0)) == INVALID
    assert _rope(rot=dict(n_axes=2), pos=dict(ld=2)) == INVALID  # two axes, no map
    assert _rope(rot=dict(pair_axis=bytes([0] * 63 + [1]))) == INVALID  # axis 1 of one
    for s in (0.0, float("nan"), float("inf")):
        assert _rope(rot=dict(scale=s)) == INVALID
    assert _rope(rot=dict(freqs=C + 2)) == ALIGN
    assert _rope(pos=dict(data=None)) == INVALID
    assert _rope(pos=dict(type=3)) == INVALID
    assert _rope(pos=dict(rows=0)) == INVALID
    assert _rope(pos=dict(rows=4)) == INVALID                   # more rows than tokens
    assert _rope(pos=dict(ld=0)) == INVALID
    assert _rope(pos=dict(type=1, data=C + 4)) == ALIGN
    assert _rope(x=(A + 1, 512, 128)) == ALIGN
    assert _rope(x=(A, -512, 128)) == INVALID
    assert _rope(y=(B, 512, 64)) == INVALID                     # heads that meet
    assert _rope(y=(B, 300, 128)) == INVALID                    # tokens that meet
    assert _rope(y=(B, 1 << 41, 128)) == INVALID
    # overlaps other than the same view
    assert _rope(y=(A + 256, 512, 128)) == INVALID
    assert _rope(y=(A, 1024, 128)) == INVALID
    assert _rope(x=(A, 512, 128), y=(A + 2 * 128, 512, 128)) == INVALID
    # column ranges of the same rows do meet here: 4 heads wide, 3 heads on, rows of 6
    assert _rope(x=(A, 768, 128), y=(A + 2 * 3 * 128, 768, 128)) == INVALID


def test_zero_tokens_do_nothing():
    assert _rope(x=(None, 512, 128), y=(None, 512, 128), tokens=0, pos=dict(data=None, rows=0)) == hsq.HSQ_OK
    assert _append(k=(None, 1024, 128), v=(None, 1024, 128), q=None, q_out=None, tokens=0) == hsq.HSQ_OK


def _append(k=(A, 1024, 128), v=(A + (1 << 16), 1024, 128), q=(A + (2 << 16), 4096, 128),
            q_out=(A + (3 << 16), 4096, 128), dtype=0, tokens=4, q_heads=32, kv=8, dim=128, rot=True, pos=None, cache=None,
            seqs=None, no=()):
    c = dict(k=B, v=C, dtype=0, pages=4, page_size=16, page_stride=16 * 1024, slot_stride=1024, head_stride=128,
             k_scale=None, v_scale=None)
    c.update(cache or {})
    s = dict(block_table=1 << 28, cache_lens=(1 << 28) + 4096, cu_seqlens=None, count=4, max_pages=5, table_ld=5)
    s.update(seqs or {})
    ref = lambda t: None if t is None else ctypes.byref(hsq._CHeads(*t))  # noqa: E731
    r = ctypes.byref(hsq._CRotation(freqs=1 << 27, pair_axis=None, pairs=64, n_axes=1, scale=1.0)) if rot else None
    p = None if pos is None else ctypes.byref(hsq._CPositions(**pos))
    return hsq.load().hsq_kv_append(ref(k), ref(v), ref(q), ref(q_out), dtype, tokens, q_heads if q else 0, kv, dim, r, p,
                                    None if "cache" in no else ctypes.byref(hsq._CPagedCache(**c)),
                                    None if "seqs" in no else ctypes.byref(hsq._CSequences(**s)), None)


def test_append_refusals():
    assert _append(no=("cache",)) == INVALID
    assert _append(no=("seqs",)) == INVALID
    assert _append(k=None) == INVALID
    assert _append(q_out=None) == INVALID
    assert _append(dtype=2) == INVALID
    assert _append(kv=0) == INVALID
    assert _append(dim=520) == UNSUP
    assert _append(cache=dict(dtype=3)) == INVALID
    assert _append(cache=dict(pages=0)) == INVALID
    assert _append(cache=dict(page_size=0)) == INVALID
    assert _append(cache=dict(k_scale=1 << 26)) == INVALID       # scales belong to an E4M3 cache
    assert _append(cache=dict(k=None)) == INVALID
    assert _append(cache=dict(k=B + 1)) == ALIGN
    assert _append(cache=dict(head_stride=64)) == INVALID        # heads that meet
    assert _append(cache=dict(slot_stride=512)) == INVALID       # slots that meet
    assert _append(cache=dict(page_stride=8 * 1024)) == INVALID  # pages that meet
    assert _append(cache=dict(page_stride=-1)) == INVALID
    assert _append(cache=dict(v=B + 4096)) == INVALID            # v inside k
    assert _append(cache=dict(v=A)) == INVALID                   # the cache over the inputs
    assert _append(seqs=dict(block_table=None)) == INVALID
    assert _append(seqs=dict(cache_lens=None)) == INVALID
    assert _append(seqs=dict(cache_lens=(1 << 28) + 2)) == ALIGN
    assert _append(seqs=dict(max_pages=0)) == INVALID
    assert _append(seqs=dict(table_ld=4)) == INVALID
    assert _append(seqs=dict(count=0)) == INVALID
    assert _append(seqs=dict(count=3)) == INVALID                # no cu_seqlens: one token per sequence
    p = dict(data=1 << 26, type=0, rows=4, ld=1)
    assert _append(rot=False, pos=p) == INVALID                  # positions without a rotation
    assert _append(pos=dict(p, rows=3)) == INVALID
    assert _append(q_out=(A, 4096, 128)) == INVALID              # q_out over k
    # (k, v and q as columns of one output, q_out in place, would be accepted: not called with fake pointers)
    assert _append(k=(A + 2 * 4096, 6144, 128), v=(A + 2 * 5120, 6144, 128), q=(A, 6144, 128),
                   q_out=(A + 2 * 1024, 6144, 128)) == INVALID


def test_bad_page_has_a_name():
    assert hsq.status_string(hsq.HSQ_ERR_BAD_PAGE) == "HSQ_ERR_BAD_PAGE"


def test_struct_layouts_match_the_header(tmp_path):
    """The binding's structures against the header's, by a C program's sizes and offsets."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    pairs = {"hsq_epilogue": hsq._CEpilogue, "hsq_heads": hsq._CHeads, "hsq_rotation": hsq._CRotation,
             "hsq_positions": hsq._CPositions, "hsq_paged_cache": hsq._CPagedCache, "hsq_sequences": hsq._CSequences}
    lines = []
    for name, c in pairs.items():
        lines.append(f'printf("%zu ", sizeof({name}));')
        lines += [f'printf("%zu ", offsetof({name}, {f}));' for f, _ in c._fields_]
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include "hsq.h"\nint main(void) {' + "\n".join(lines) + "return 0;}\n")
    exe = str(tmp_path / "t")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), "-I", "/usr/local/cuda/include", "-o", exe, str(src)],
                   check=True)
    got = [int(v) for v in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for c in pairs.values():
        want.append(ctypes.sizeof(c))
        want += [getattr(c, f).offset for f, _ in c._fields_]
    assert got == want
    # ... and what the two calls pack themselves
    packed = {hsq._HEADS: hsq._CHeads, hsq._POSITIONS: hsq._CPositions, hsq._PAGED_CACHE: hsq._CPagedCache,
              hsq._SEQUENCES: hsq._CSequences}
    for st, c in packed.items():
        assert st.size == ctypes.sizeof(c)
        n = len(c._fields_)
        got = c.from_buffer_copy(st.pack(*range(1, n + 1)))
        assert [getattr(got, f) for f, _ in c._fields_] == list(range(1, n + 1))
