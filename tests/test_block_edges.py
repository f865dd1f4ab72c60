"""Host-side checks of the calls around a linear that need no GPU: overlaps, counts and
devices that are refused before anything is launched, and the binding's objects."""
import ctypes

import pytest
import torch

from w4a4_rank_assisted_b200 import hsq

A, FAR = 1 << 20, 1 << 30   # fake device addresses: every call below has to be refused before they are touched
INVALID = hsq.HSQ_ERR_INVALID_ARG


@pytest.mark.parametrize("M,r,group", [(1, 4, 64), (2, 0, 128), (4, 1, 64)])
@pytest.mark.parametrize("shift", [0, 64, -64], ids=["same", "above", "below"])
def test_the_stream_form_refuses_y_over_x(M, r, group, shift):
    """With an epilogue, without one, and through one that asks for nothing: its blocks read X while others write Y."""
    lib = hsq.load()
    assert hsq.hsq_fused_form(M, 128, 128, r, group) == 1
    low = None if r == 0 else FAR
    args = (A, FAR, low, FAR, FAR, low, None, M, 128, 128, r, group, A + shift, 0)
    assert lib.hsq_linear_forward_fused(*args, None) == INVALID
    assert lib.hsq_linear_forward_fused_ep(*args, None, None) == INVALID
    assert lib.hsq_linear_forward_fused_ep(*args, ctypes.byref(hsq._CEpilogue()), None) == INVALID
    assert lib.hsq_linear_forward_fused_ep(*args, ctypes.byref(hsq._CEpilogue(act=4)), None) == INVALID


class FakeTensor:
    """What the binding asks of a CUDA tensor, without a GPU."""

    is_cuda = True

    def __init__(self, device, *shape, dtype=torch.bfloat16):
        self.device_index, self.shape, self.dtype = device, torch.Size(shape), dtype

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        s = tuple(self.shape[j + 1:].numel() for j in range(len(self.shape)))
        return s if i is None else s[i]

    address = FAR

    def data_ptr(self):
        return self.address


class FakeLibrary:
    """Records every call with the device that is current during it."""

    def __init__(self, current):
        self.calls, self.args, self.current = [], None, current

    def __getattr__(self, name):
        def call(*a):
            self.calls.append((name, self.current[-1], a[-1]))
            self.args = a
            return 0
        return call

    def struct(self, kind, i):
        """Argument i of the last call, as the C structure that it points to."""
        a = self.args[i]
        return kind.from_buffer_copy(a if isinstance(a, bytes) else bytes(a._obj))


@pytest.fixture
def library(monkeypatch):
    """The fake library with device 0 current; device d's current stream is 100 + d."""
    current = [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *e):
            current.pop()

    lib = FakeLibrary(current)
    monkeypatch.setattr(hsq, "load", lambda *a: lib)
    monkeypatch.setattr(hsq, "_raw_stream", lambda d: 100 + d)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "device", Device)
    return lib


def _tensors(device, names):
    return {n: FakeTensor(device, 16, 64) for n in names}


CALLS = {
    "hsq_linear_forward_ep": ("x_codes", "x_scales", "U", "w_codes", "w_scales", "w_e4m3", "L2", "bias", "workspace"),
    "hsq_linear_forward_noalloc_ep": ("x_codes", "x_scales", "U", "w_codes", "w_scales", "L2", "bias"),
    "hsq_linear_forward_x_ep": ("X", "s", "L1", "w_codes", "w_scales", "w_e4m3", "L2", "bias", "workspace"),
    "hsq_linear_forward_fused_ep": ("X", "s", "L1", "w_codes", "w_scales", "L2", "bias"),
    "hsq_fp4_linear_forward_ep": ("x_codes", "x_sf", "x_gs", "U", "w_codes", "w_sf", "w_gs", "L2", "bias"),
}


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_of_a_forward_lives_on_its_device(name, library):
    """One tensor on another GPU refuses the call; all of them on another GPU than the current one run there."""
    call = getattr(hsq, name)
    dims = dict(M=16, N=64, K=64, r=4)
    for other in CALLS[name]:
        t = _tensors(0, CALLS[name])
        t[other] = FakeTensor(1, 16, 64)
        with pytest.raises(ValueError, match="device"):
            call(Y=FakeTensor(0, 16, 64), epilogue=None, **t, **dims)
    assert not library.calls
    call(Y=FakeTensor(1, 16, 64), epilogue=None, **_tensors(1, CALLS[name]), **dims)
    assert library.calls == [(name, 1, 101)]


class Parts:
    def __init__(self, device, **kw):
        self.__dict__.update(_tensors(device, ("w_codes", "w_scales", "w_e4m3", "L1", "L2", "bias", "s", "w_sf", "w_gs",
                                               "x_codes", "x_scales", "x_sf", "x_gs", "U")), N=64, K=64, r=4, group=64, **kw)


@pytest.mark.parametrize("fp4", [False, True], ids=["int4", "nvfp4"])
def test_both_steps_of_a_forward_run_on_its_tensors_device(fp4, library):
    """With an epilogue the activation step, too, runs on the tensors' device, and is not launched where the forward
    would be refused."""
    f = hsq.fp4_forward if fp4 else hsq.forward
    names = ["hsq_fp4_quantize_act", "hsq_fp4_linear_forward_ep"] if fp4 else ["hsq_quantize_act", "hsq_linear_forward_ep"]
    f(Parts(1), FakeTensor(1, 16, 64), Parts(1), FakeTensor(1, 16, 64), epilogue=hsq.Epilogue("silu"))
    assert [c[:2] for c in library.calls] == [(n, 1) for n in names] and {c[2] for c in library.calls} == {101}
    library.calls.clear()
    f(Parts(1), FakeTensor(1, 16, 64), Parts(1), FakeTensor(1, 16, 64), epilogue=hsq.Epilogue("silu"), stream=7)
    assert [c[1:] for c in library.calls] == [(1, 7)] * 2
    library.calls.clear()
    for X, Y, layer, act in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0)):
        with pytest.raises(ValueError, match="device"):
            f(Parts(layer), FakeTensor(X, 16, 64), Parts(act), FakeTensor(Y, 16, 64), epilogue=hsq.Epilogue("silu"))
    with pytest.raises(ValueError):
        f(Parts(1), FakeTensor(1, 16, 64), Parts(1), FakeTensor(1, 16, 72), epilogue=hsq.Epilogue("silu"))
    assert not library.calls


def test_append_refuses_more_head_blocks_than_a_grid_holds():
    """196608 heads of 447 single elements' units: refused as an argument, not by the launch.  65537 of a kind: never
    taken."""
    far, ref, H = 1 << 44, ctypes.byref, 65536

    def append(q_heads, kv, dim=511):
        at = lambda i: hsq._CHeads((i + 1) * far, H * dim, dim)  # noqa: E731
        cache = hsq._CPagedCache(k=5 * far, v=6 * far, dtype=0, pages=2, page_size=4, page_stride=4 * H * dim,
                                 slot_stride=H * dim, head_stride=dim)
        seqs = hsq._CSequences(block_table=7 * far, cache_lens=8 * far, cu_seqlens=None, count=1, max_pages=2, table_ld=2)
        rot = hsq._CRotation(freqs=9 * far, pair_axis=None, pairs=64, n_axes=1, scale=1.0)
        return hsq.load().hsq_kv_append(ref(at(0)), ref(at(1)), ref(at(2)), ref(at(3)), 0, 1, q_heads, kv, dim, ref(rot),
                                        None, ref(cache), ref(seqs), None)

    assert append(H, H) == hsq.HSQ_ERR_UNSUPPORTED
    assert append(1, H) == hsq.HSQ_ERR_UNSUPPORTED  # 131073 heads, 65537 blocks
    assert append(H + 1, 1) == INVALID and append(1, H + 1) == INVALID


def test_a_decode_step_of_no_sequences_does_nothing():
    """One new token per sequence and no sequence: tokens == count == 0."""
    ref = ctypes.byref
    heads = hsq._CHeads(None, 512, 128)
    cache = hsq._CPagedCache(k=A, v=FAR, dtype=0, pages=2, page_size=4, page_stride=4 * 512, slot_stride=512, head_stride=128)
    call = lambda tokens, **kw: hsq.load().hsq_kv_append(  # noqa: E731
        ref(heads), ref(heads), None, None, 0, tokens, 0, 4, 128, None, None, ref(cache),
        ref(hsq._CSequences(**{**dict(count=0, max_pages=2, table_ld=2), **kw})), None)
    assert call(0) == hsq.HSQ_OK
    assert call(0, count=-1) == INVALID
    assert call(1) == INVALID
    assert call(0, cu_seqlens=A) == INVALID  # cu_seqlens of no sequence


def _relu_x(Y, epilogue):
    """hsq_linear_forward_x_ep on 16 x 64 fakes (its epilogue is argument -4)."""
    names = CALLS["hsq_linear_forward_x_ep"]
    hsq.hsq_linear_forward_x_ep(Y=Y, epilogue=epilogue, M=16, N=64, K=64, r=4, **_tensors(0, names))


@pytest.mark.parametrize("rows,want", [(1, 1), (4, 4), (16, 16), (1 << 31, 16), ((1 << 32) + 1, 16), ((1 << 40) + 4, 16)])
def test_mul_rows_of_any_size(rows, want, library):
    """A row count beyond an int says the same as one of the token count: it may not come out smaller."""
    mul = FakeTensor(0, -(-16 // rows), 64)
    _relu_x(FakeTensor(0, 16, 64), hsq.Epilogue("relu", mul=mul, mul_rows=rows))
    assert -(-16 // library.struct(hsq._CEpilogue, -4).mul_rows) == -(-16 // want)


def test_an_epilogue_reads_its_tensors_where_they_are(library):
    """A tensor whose storage was replaced (as a module's .to() and .data do) since the epilogue was made."""
    mul, res, Y = FakeTensor(0, 16, 64), FakeTensor(0, 16, 64), FakeTensor(0, 16, 64)
    ep = hsq.Epilogue("silu", mul=mul, residual=res)
    _relu_x(Y, ep)
    mul.address, res.address, res.dtype = 3 * FAR, 4 * FAR, torch.float32
    _relu_x(Y, ep)
    c = library.struct(hsq._CEpilogue, -4)
    assert (c.act, c.mul, c.mul_dtype, c.mul_rows, c.mul_ld) == (4, 3 * FAR, 0, 1, 64)
    assert (c.residual, c.residual_dtype, c.residual_ld) == (4 * FAR, 1, 64)
    res.dtype = torch.float16
    with pytest.raises(ValueError):
        _relu_x(Y, ep)


def test_a_rotation_reads_its_frequencies_where_they_are(library):
    f = FakeTensor(0, 32, dtype=torch.float32)
    rot = hsq.Rotation(f, [0, 1] * 16, interleaved=True, transpose=True, scale=0.5)
    f.address = 5 * FAR
    x, y, pos = FakeTensor(0, 3, 2, 64), FakeTensor(0, 3, 2, 64), FakeTensor(0, 3, 2, dtype=torch.int32)
    hsq.hsq_rope(x, y, pos, rot)
    c = library.struct(hsq._CRotation, 6)
    assert (c.freqs, c.pairs, c.n_axes, c.interleaved, c.transpose, c.scale) == (5 * FAR, 32, 2, 1, 1, 0.5)
    at = hsq._CRotation.pair_axis.offset
    assert ctypes.string_at(int.from_bytes(bytes(c)[at:at + 8], "little"), 32) == bytes([0, 1] * 16)
    f.dtype = torch.float64
    with pytest.raises(ValueError):
        hsq.hsq_rope(x, y, pos, rot)
    f.dtype, f.shape = torch.float32, torch.Size((16,))
    with pytest.raises(ValueError):
        hsq.hsq_rope(x, y, pos, rot)


def test_the_packed_epilogue_is_the_structure():
    assert hsq._EPILOGUE.size == ctypes.sizeof(hsq._CEpilogue)
    got = hsq._CEpilogue.from_buffer_copy(hsq._EPILOGUE.pack(*range(1, 9)))
    assert [getattr(got, n) for n, _ in hsq._CEpilogue._fields_] == list(range(1, 9))
