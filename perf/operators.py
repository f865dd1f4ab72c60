"""Cases that time the operators around a packed linear layer, and their plain forms.

Three operators, as one transformer block uses them in turn:

- ``linear``: the W4A4 (or NVFP4) linear with its epilogue,
  ``Y = act(X_hat Q(R)^T + U L2 + b) * mul + residual``;
- ``rope``: the rotation of the query and key heads of a fused projection by
  positions with one or more axes, and its transpose (its gradient);
- ``append``: keys rotated and written with their values into a paged cache,
  queries rotated on the way.

``run`` computes them in elementary torch operations, or, with ``own`` set,
through the library's calls.
"""
import math
import random

import torch

#: set by whoever imports the file: False computes the plain forms, True calls the library
own = False

DEV = "cuda"
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64,
          "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------- cases
def listed():
    lin = {"op": "linear", "fmt": "int4", "group": 64, "r": 4, "bias": False, "act": "none", "mul": "none",
           "residual": False, "out": "bf16"}
    rope = {"op": "rope", "dtype": "bf16", "transpose": False, "scale": 1.0, "pos": "i32"}
    app = {"op": "append", "dtype": "bf16", "cache": "bf16", "layout": "slots", "interleaved": False, "rotate": True}
    return [
        # one new token of a gated MLP: silu(gate) * up in the gate projection's own launch
        {**lin, "name": "linear_decode1_silu_mul", "M": 1, "K": 4096, "N": 12288, "act": "silu", "mul": "full"},
        # sixteen sequences decoding: the MLP's way back, added onto the residual stream
        {**lin, "name": "linear_decode16_residual", "M": 16, "K": 12288, "N": 4096, "group": 128, "residual": True},
        # an image transformer's first MLP layer with its GELU, 4096 latent tokens
        {**lin, "name": "linear_mlp_up_gelu", "M": 4096, "K": 1152, "N": 4608, "bias": True, "act": "gelu_tanh"},
        # a ragged batch with a gate per sample, rank 32, on an fp32 residual stream
        {**lin, "name": "linear_gated_residual_f32", "M": 997, "K": 5600, "N": 2240, "r": 32, "bias": True,
         "mul": "sample", "residual": True, "out": "f32"},
        # a long prefill's gate projection
        {**lin, "name": "linear_prefill_silu_mul", "M": 8192, "K": 4096, "N": 12288, "group": 128, "act": "silu",
         "mul": "full"},
        # the NVFP4 form: an MLP's way back with its gate and residual
        {**lin, "name": "linear_nvfp4_gated_residual", "fmt": "nvfp4", "M": 4096, "K": 4608, "N": 1152, "bias": True,
         "mul": "sample", "residual": True},
        # one new token: 32 query and 8 key heads of one fused projection
        {**rope, "name": "rope_decode1", "tokens": 1, "heads": 40, "dim": 128, "axes": 1, "pairs": 64,
         "interleaved": False, "pos_rows": 1, "wide": 48},
        # an image and its text, 4608 tokens, three axes, 24 query and 24 key heads inside the fused projection
        {**rope, "name": "rope_image_3axes", "tokens": 4608, "heads": 48, "dim": 128, "axes": 3, "pairs": 64,
         "interleaved": True, "pos": "f32", "pos_rows": 4608, "wide": 72},
        # gradient of a video's queries, two clips that share their positions, partly rotated heads, fp32
        {**rope, "name": "rope_video_gradient_f32", "tokens": 15606, "heads": 16, "dim": 80, "axes": 3, "pairs": 32,
         "interleaved": False, "pos": "i64", "pos_rows": 7803, "wide": 16, "dtype": "f32", "transpose": True,
         "scale": 1.25},
        # one sequence, one new token, a long way in
        {**app, "name": "append_decode1", "seqs": 1, "new": 1, "pad": 0, "context": 100000, "page": 16, "q": 32,
         "kv": 8, "dim": 128},
        # a full decode batch, one token each, into an FP8 cache
        {**app, "name": "append_decode256_e4m3", "seqs": 256, "new": 1, "pad": 0, "context": 3000, "page": 16, "q": 32,
         "kv": 8, "dim": 128, "cache": "e4m3"},
        # prompts of many lengths, packed, that end inside pages; head-major pages
        {**app, "name": "append_prefill_ragged", "seqs": 13, "new": 630, "pad": 37, "context": 200, "page": 64, "q": 32,
         "kv": 8, "dim": 128, "layout": "heads"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(("linear", "linear", "rope", "append"))
    if op == "linear":
        while True:
            c = {"op": op, "fmt": rng.choice(("int4", "int4", "nvfp4")), "group": rng.choice((64, 128)),
                 "r": rng.choice((0, 1, 4, 5, 16, 32)), "bias": rng.random() < 0.5,
                 "act": rng.choice(("none", "relu", "gelu_tanh", "gelu_erf", "silu")),
                 "mul": rng.choice(("none", "full", "sample")), "residual": rng.random() < 0.5,
                 "out": rng.choice(("bf16", "bf16", "f32")), "M": _log(rng, 1, 8192), "K": 8 * _log(rng, 32, 1536),
                 "N": 8 * _log(rng, 32, 1536)}
            if c["M"] * c["K"] * c["N"] <= 2 ** 38:
                return c
    if op == "rope":
        while True:
            dim = rng.choice((32, 64, 72, 80, 96, 128, 128, 160, 256))
            rows = _log(rng, 1, 32768)
            heads = _log(rng, 1, 64)
            c = {"op": op, "dtype": rng.choice(("bf16", "bf16", "f32")), "transpose": rng.random() < 0.4,
                 "scale": rng.choice((1.0, 1.0, 0.875)), "pos": rng.choice(("i32", "i64", "f32")),
                 "tokens": rows * rng.choice((1, 1, 2, 3)), "heads": heads, "dim": dim, "axes": rng.randint(1, 4),
                 "pairs": rng.choice((dim // 2, dim // 2, dim // 4)), "interleaved": rng.random() < 0.5,
                 "pos_rows": rows, "wide": heads + rng.choice((0, 0, 1, 8))}
            if c["tokens"] * c["wide"] * dim <= 2 ** 26:
                return c
    while True:
        kv = rng.choice((1, 2, 4, 8, 8, 16))
        c = {"op": op, "dtype": rng.choice(("bf16", "bf16", "f32")), "cache": rng.choice(("bf16", "e4m3", "f32")),
             "layout": rng.choice(("slots", "heads")), "interleaved": rng.random() < 0.3, "rotate": rng.random() < 0.85,
             "seqs": _log(rng, 1, 256), "new": rng.choice((1, 1, _log(rng, 1, 2000))), "pad": rng.choice((0, 0, 5)),
             "context": _log(rng, 1, 4000), "page": rng.choice((1, 8, 16, 24, 32, 64, 128)), "q": kv * rng.choice((1, 4, 7)),
             "kv": kv, "dim": rng.choice((64, 72, 80, 128, 128, 256))}
        if c["new"] == 1:
            c["pad"] = 0
        if c["seqs"] * c["new"] * (c["q"] + 2 * kv) * c["dim"] <= 2 ** 26 and \
                c["seqs"] * (c["new"] + c["context"] + c["page"]) * kv * c["dim"] <= 2 ** 28:
            return c


# ---------------------------------------------------------------- inputs
def _codes(g, rows, K, group):
    """Packed INT4 codes and group-major scales of a Gaussian matrix (the stored form of a residual)."""
    Kp = -(-K // group) * group
    w = torch.zeros(rows, Kp, device=DEV)
    w[:, :K] = torch.randn(rows, K, generator=g, device=DEV) * 0.02
    w = w.view(rows, -1, group)
    sc = w.abs().amax(2) / 7.0
    q = torch.where(sc[..., None] > 0, torch.round(w / sc[..., None]), torch.zeros_like(w)).clamp_(-7, 7)
    q = q.to(torch.int32).view(rows, Kp) & 15
    packed = (q[:, 0::2] | (q[:, 1::2] << 4)).to(torch.uint8).contiguous()
    ld = -(-rows // 4) * 4
    scales = torch.zeros(sc.shape[1], ld, device=DEV)
    scales[:, :rows] = sc.t()
    return packed, scales


def _fp4_weights(g, rows, K):
    """Random NVFP4 weights: packed E2M1 codes, E4M3 block scales in 128 x 64 atoms, the tensor scale."""
    Kq = -(-K // 64) * 64
    q = torch.randint(0, 16, (rows, Kq), generator=g, device=DEV, dtype=torch.int32)
    q = torch.where(q == 8, torch.zeros_like(q), q)  # a zero has code 0
    q[:, K:] = 0
    packed = (q[:, 0::2] | (q[:, 1::2] << 4)).to(torch.uint8).contiguous()
    sf = (32 + 200 * torch.rand(rows, Kq // 16, generator=g, device=DEV)).to(torch.float8_e4m3fn).view(torch.uint8)
    sf[:, -(-K // 16):] = 0
    pad = torch.zeros(-(-rows // 128) * 128, Kq // 16, device=DEV, dtype=torch.uint8)
    pad[:rows] = sf
    atoms = pad.view(-1, 4, 32, Kq // 64, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    gs = torch.tensor([0.06 / 2688, 0.0, 0.0, 0.0], device=DEV)
    return packed, atoms, gs


def _prepare_linear(c, g):
    M, K, N, r = c["M"], c["K"], c["N"], c["r"]
    bf = torch.bfloat16
    X = torch.randn(M, K, generator=g, device=DEV)
    X[:, torch.randperm(K, generator=g, device=DEV)[:max(1, K // 200)]] *= 30.0  # a few outlier channels
    X = X.to(bf)
    s = (X.float().abs().amax(0).clamp_min(1e-3) / 0.08).sqrt()
    out = _TYPES[c["out"]]
    st = {"case": c, "X": X, "s": s, "L1": None, "L2": None, "bias": None, "mul": None, "residual": None,
          "mul_rows": 1, "Y": torch.empty(M, N, dtype=out, device=DEV)}
    if r:
        st["L1"] = (torch.randn(K, r, generator=g, device=DEV) * 0.02).to(bf)
        st["L2"] = (torch.randn(r, N, generator=g, device=DEV) * 0.02).to(bf)
    if c["bias"]:
        st["bias"] = (torch.randn(N, generator=g, device=DEV) * 0.5).to(bf)
    if c["mul"] == "full":
        st["mul"] = torch.randn(M, N, generator=g, device=DEV).to(bf)
    elif c["mul"] == "sample":  # one of the modulation vectors of every sample: a column range of a wider tensor
        st["mul_rows"] = -(-M // 2)
        st["mul"] = torch.randn(-(-M // st["mul_rows"]), 2 * N, generator=g, device=DEV).to(bf)[:, N:]
    if c["residual"]:
        st["residual"] = torch.randn(M, N, generator=g, device=DEV).to(out)
    if c["fmt"] == "int4":
        st["w_codes"], st["w_scales"] = _codes(g, N, K, c["group"])
    else:
        st["w_codes"], st["w_sf"], st["w_gs"] = _fp4_weights(g, N, K)
    return st


def _freqs(pairs, axes):
    """Frequencies and axes of the pairs: the axes take consecutive runs, each with its own ladder."""
    n = [pairs // axes + (1 if a < pairs % axes else 0) for a in range(axes)]
    f = torch.cat([10000.0 ** (-torch.arange(k, dtype=torch.float64) / max(k, 1)) for k in n])
    return f.float().to(DEV), [a for a, k in enumerate(n) for _ in range(k)]


def _prepare_rope(c, g):
    dt = _TYPES[c["dtype"]]
    x = torch.randn(c["tokens"], c["wide"], c["dim"], generator=g, device=DEV).to(dt)[:, :c["heads"]]
    y = torch.zeros(c["tokens"], c["heads"], c["dim"], device=DEV, dtype=dt)
    freqs, axes = _freqs(c["pairs"], c["axes"])
    far = torch.tensor([4096.0, 300.0, 300.0, 64.0])[:c["axes"]].to(DEV)
    pos = torch.rand(c["pos_rows"], c["axes"], generator=g, device=DEV) * far
    pos = pos.to(_TYPES[c["pos"]]) if c["pos"] != "f32" else pos.floor() * 0.5
    return {"case": c, "x": x, "y": y, "freqs": freqs, "axes": axes, "pos": pos.contiguous(),
            "axis_of": torch.tensor(axes, device=DEV)}


def _lengths(c):
    """New tokens and tokens already cached of each sequence: the case's own."""
    r = random.Random(c["seqs"] * 1000003 + c["new"] * 1009 + c["context"])
    n_new = [1] * c["seqs"] if c["new"] == 1 else [int(c["new"] * r.uniform(0.0, 2.0)) for _ in range(c["seqs"])]
    return n_new, [int(c["context"] * r.uniform(0.0, 2.0)) for _ in range(c["seqs"])]


def _prepare_append(c, g):
    dt, ct = _TYPES[c["dtype"]], _TYPES[c["cache"]]
    B, kv, q, D, ps = c["seqs"], c["kv"], c["q"], c["dim"], c["page"]
    n_new, lens = _lengths(c)
    real = sum(n_new)
    T = max(1, real + c["pad"])
    cols = max(-(-(a + b) // ps) for a, b in zip(lens, n_new)) + 1
    # only the pages that this call writes differ between sequences; the ones before are a shared pool
    first = [a // ps for a in lens]
    need = [max(0, -(-(a + b) // ps) - f) for a, b, f in zip(lens, n_new, first)]
    pages = sum(need) + 8
    perm = (torch.randperm(pages - 8, generator=g, device=DEV) + 8).tolist() if pages > 8 else []
    rows = []
    for f, k in zip(first, need):
        mine, perm = perm[:k], perm[k:]
        rows.append([i % 8 for i in range(f)] + mine + [-1] * (cols - f - k))
    shape = (pages, ps, kv, D) if c["layout"] == "slots" else (pages, kv, ps, D)
    caches = [torch.randn(shape, generator=g, device=DEV).to(ct) for _ in range(2)]
    if c["layout"] == "heads":
        caches = [t.transpose(1, 2) for t in caches]
    qkv = torch.randn(T, q + 2 * kv, D, generator=g, device=DEV).to(dt)
    cu = [0]
    for k in n_new:
        cu.append(cu[-1] + k)
    freqs, axes = _freqs(D // 2, 1)
    as_int = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    scale = [0.01 + 0.02 * torch.rand(kv, generator=g, device=DEV) for _ in range(2)] if c["cache"] == "e4m3" else [None] * 2
    return {"case": c, "q": qkv[:, :q], "k": qkv[:, q:q + kv], "v": qkv[:, q + kv:], "k_cache": caches[0],
            "v_cache": caches[1], "q_out": torch.zeros(T, q, D, device=DEV, dtype=dt), "table": as_int(rows),
            "lens": as_int(lens), "cu": None if c["new"] == 1 else as_int(cu), "real": real, "freqs": freqs,
            "k_scale": scale[0], "v_scale": scale[1]}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    st = {"linear": _prepare_linear, "rope": _prepare_rope, "append": _prepare_append}[case["op"]](dict(case), g)
    if own:
        st["handle"] = _linear_handle(st) if case["op"] == "linear" else _rotation(st)
    return st


# ---------------------------------------------------------------- the library's calls
def _linear_handle(st):
    """What a program keeps of a layer between calls: its workspace, and for many tokens the expanded weights."""
    from w4a4_rank_assisted_b200 import hsq
    c = st["case"]
    h = {"epilogue": hsq.Epilogue(c["act"], mul=st["mul"], mul_rows=st["mul_rows"], residual=st["residual"])}
    if c["fmt"] == "nvfp4":
        h["act"] = hsq.Fp4ActBuffers(c["M"], c["K"], c["r"], DEV)
    elif not hsq.fused_supported(c["M"], c["K"], c["r"], c["group"], N=c["N"]):
        h["w_e4m3"] = None
        if c["M"] > 64:
            h["w_e4m3"] = torch.empty(hsq.hsq_weights_e4m3_bytes(c["N"], c["K"], c["group"]), dtype=torch.uint8, device=DEV)
            hsq.hsq_expand_weights(st["w_codes"], c["N"], c["K"], h["w_e4m3"], group=c["group"])
        n = hsq.hsq_workspace_bytes_x(c["M"], c["N"], c["K"], c["r"], c["group"], h["w_e4m3"] is not None)
        h["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    return h


def _rotation(st):
    """What a program keeps of its rotation between calls."""
    from w4a4_rank_assisted_b200 import hsq
    c = st["case"]
    if not c.get("rotate", True):
        return None
    return hsq.Rotation(st["freqs"], st.get("axes"), interleaved=c["interleaved"], transpose=c.get("transpose", False),
                        scale=c.get("scale", 1.0))


def _own_linear(st):
    from w4a4_rank_assisted_b200 import hsq
    c, h, Y = st["case"], st["handle"], st["Y"]
    M, N, K, r = c["M"], c["N"], c["K"], c["r"]
    out = hsq.HSQ_OUT_F32 if c["out"] == "f32" else hsq.HSQ_OUT_BF16
    if c["fmt"] == "nvfp4":
        a = h["act"]
        hsq.hsq_fp4_quantize_act(st["X"], st["s"], st["L1"], M, K, r, a.x_codes, a.x_sf, a.x_gs, a.U)
        hsq.hsq_fp4_linear_forward_ep(a.x_codes, a.x_sf, a.x_gs, a.U, st["w_codes"], st["w_sf"], st["w_gs"], st["L2"],
                                      st["bias"], M, N, K, r, Y, h["epilogue"], out=out)
    elif "ws" in h:
        hsq.hsq_linear_forward_x_ep(st["X"], st["s"], st["L1"], st["w_codes"], st["w_scales"], h["w_e4m3"], st["L2"],
                                    st["bias"], M, N, K, r, Y, h["epilogue"], out=out, workspace=h["ws"],
                                    ws_bytes=h["ws"].numel(), group=c["group"])
    else:
        hsq.hsq_linear_forward_fused_ep(st["X"], st["s"], st["L1"], st["w_codes"], st["w_scales"], st["L2"],
                                        st["bias"], M, N, K, r, Y, h["epilogue"], out=out, group=c["group"])
    return Y


def _own_rope(st):
    from w4a4_rank_assisted_b200 import hsq
    hsq.hsq_rope(st["x"], st["y"], st["pos"], st["handle"])
    return st["y"]


def _own_append(st):
    from w4a4_rank_assisted_b200 import hsq
    hsq.hsq_kv_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["lens"], cu_seqlens=st["cu"],
                      rotation=st["handle"], q=st["q"], q_out=st["q_out"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


# ---------------------------------------------------------------- the plain forms
def _unpack(p):
    q = torch.stack((p & 15, p >> 4), dim=2).reshape(p.shape[0], -1)
    return q


def _signed(p):
    q = _unpack(p).to(torch.float32)
    return torch.where(q > 7, q - 16, q)


def _e2m1_value(code):
    m = (code & 7).float()
    v = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2, 2 * m - 8))  # 0 .5 1 1.5 | 2 3 | 4 6
    return torch.where((code & 8) > 0, -v, v)


def _e2m1_round(v):
    """The nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the even mantissa), with v's sign."""
    a = v.abs()
    q = 0.5 * ((a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) + 1.0 * ((a > 2.5).float() + (a >= 3.5)) + 2.0 * (a > 5.0)
    return q * torch.sign(v)


def _block_scales(atoms, rows, KC):
    sf = atoms.view(-1, KC, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4 * KC)[:rows]
    return sf.contiguous().view(torch.float8_e4m3fn).float()


def _full(v):
    """A constant on the device: torch multiplies by the reciprocal of a host scalar instead of dividing by it."""
    return torch.full((), v, device=DEV)


def _padded(x, to):
    return x if x.shape[1] == to else torch.nn.functional.pad(x, (0, to - x.shape[1]))


def _act(y, name):
    if name == "relu":
        return torch.where(y < 0, torch.zeros_like(y), y)
    if name == "silu":
        return y / (1 + torch.exp(-y))
    if name == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if name == "gelu_erf":
        return 0.5 * y * torch.erfc(-y * math.sqrt(0.5))
    return y


def _plain_linear(st):
    c = st["case"]
    M, K, N = c["M"], c["K"], c["N"]
    xh = st["X"].float() / st["s"]
    if c["fmt"] == "int4":
        grp = c["group"]
        G = -(-K // grp)
        xg = _padded(xh, G * grp).view(M, G, grp)
        sc = xg.abs().amax(2, keepdim=True) / _full(7.0)
        xq = torch.where(sc > 0, torch.round(xg / sc), torch.zeros_like(xg)).clamp_(-7, 7) * sc
        w = _signed(st["w_codes"]).view(N, G, grp) * st["w_scales"][:, :N].t()[..., None]
        y = xq.view(M, -1) @ w.view(N, -1).t()
    else:
        KC = -(-K // 64)
        xb = _padded(xh, 64 * KC).view(M, -1, 16)
        gx = xb.abs().amax() / _full(2688.0)
        b = (xb.abs().amax(2, keepdim=True) / (6.0 * gx)).clamp_max(448.0).to(torch.float8_e4m3fn).float()
        step = b * gx
        xq = torch.where(step > 0, _e2m1_round(xb / step), torch.zeros_like(xb)) * b
        w = _e2m1_value(_unpack(st["w_codes"])).view(N, -1, 16) * _block_scales(st["w_sf"], N, KC)[..., None]
        y = (xq.view(M, -1) @ w.view(N, -1).t()) * (gx * st["w_gs"][0])
    if c["r"]:
        y = y + (xh @ st["L1"].float()) @ st["L2"].float()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    y = _act(y, c["act"])
    if st["mul"] is not None:
        m = st["mul"].float()
        y = y * (m if c["mul"] == "full" else m.repeat_interleave(st["mul_rows"], 0)[:M])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(_TYPES[c["out"]])


def _rotate(x, angle, interleaved, scale):
    """x [T, H, D] fp32 rotated by angle [T, P] (fp64: positions may be far); the rest of D unchanged."""
    cos = (torch.cos(angle) * scale).float()[:, None]
    sin = (torch.sin(angle) * scale).float()[:, None]
    P = angle.shape[1]
    if interleaved:
        a, b = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
        rot = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = x[..., :P], x[..., P:2 * P]
        rot = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((rot, x[..., 2 * P:]), dim=-1)


def _plain_rope(st):
    c, x = st["case"], st["x"]
    angle = st["pos"].double()[:, st["axis_of"]] * st["freqs"].double()
    angle = angle.repeat(c["tokens"] // c["pos_rows"], 1)
    if c["transpose"]:
        angle = -angle
    return _rotate(x.float(), angle, c["interleaved"], c["scale"]).to(x.dtype)


def _plain_append(st):
    c, n = st["case"], st["real"]
    t = torch.arange(n, device=DEV)
    if st["cu"] is None:
        seq, at = t, st["lens"].long()
    else:
        cu = st["cu"].long()
        seq = (t[:, None] >= cu[None, 1:]).sum(1)
        at = st["lens"].long()[seq] + t - cu[seq]
    q, k, v = st["q"][:n].float(), st["k"][:n].float(), st["v"][:n].float()
    if c["rotate"]:
        angle = at.double()[:, None] * st["freqs"].double()
        q, k = _rotate(q, angle, c["interleaved"], 1.0), _rotate(k, angle, c["interleaved"], 1.0)
    page = st["table"].long()[seq, torch.div(at, c["page"], rounding_mode="floor")]
    slot = at % c["page"]
    for x, cache, scale in ((k, st["k_cache"], st["k_scale"]), (v, st["v_cache"], st["v_scale"])):
        if scale is not None:
            x = (x / scale[:, None]).clamp(-448.0, 448.0)
        if cache.dtype == torch.float8_e4m3fn:
            cache.view(torch.uint8)[page, slot] = x.to(cache.dtype).view(torch.uint8)
        else:
            cache[page, slot] = x.to(cache.dtype)
    st["q_out"][:n] = q.to(st["q_out"].dtype)
    return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _own_linear, "rope": _own_rope, "append": _own_append}[op](state)
    return {"linear": _plain_linear, "rope": _plain_rope, "append": _plain_append}[op](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    size = {"bf16": 2, "f32": 4, "e4m3": 1, "i32": 4, "i64": 8}
    if c["op"] == "linear":
        M, K, N, r = c["M"], c["K"], c["N"], c["r"]
        scales = N * K / 16 if c["fmt"] == "nvfp4" else 4.0 * N * -(-K // c["group"])
        b = 2.0 * M * K + 4 * K + N * K / 2 + scales + 2.0 * r * (K + N) + (2 * N if c["bias"] else 0)
        b += size[c["out"]] * M * N * (2 if c["residual"] else 1)
        b += {"none": 0, "full": 2.0 * M * N, "sample": 4.0 * N}[c["mul"]]
        return {"bytes": b, "flops": 2.0 * M * N * K + 2.0 * M * r * (K + N)}
    if c["op"] == "rope":
        n = float(c["tokens"]) * c["heads"]
        b = 2 * n * c["dim"] * size[c["dtype"]] + size[c["pos"]] * c["pos_rows"] * c["axes"] + 4 * c["pairs"]
        return {"bytes": b, "flops": 6 * n * c["pairs"]}
    n = float(sum(_lengths(c)[0]))
    b = n * c["dim"] * (size[c["dtype"]] * (2 * c["q"] + 2 * c["kv"]) + size[c["cache"]] * 2 * c["kv"]) + 12 * c["seqs"] + 4
    return {"bytes": b, "flops": n * c["dim"] * 3 * (c["q"] + c["kv"])}


# ---------------------------------------------------------------- the definitions in 64 bits
def _f32_quotient(a, b):
    """The fp32 quotient of fp32 values: rounded once (a 53-bit quotient rounded to 24 bits is the 24-bit one)."""
    return (a.double() / b.double()).float()


def _exact_linear(c, seed):
    st = prepare(c, seed)
    M, N, K = c["M"], c["N"], c["K"]
    x32 = _f32_quotient(st["X"], st["s"][None])  # the layer's definition rounds here
    x = x32.double()
    y = torch.zeros(M, N, dtype=torch.float64, device=DEV)
    nib = torch.stack([st["w_codes"].to(torch.int64) % 16, st["w_codes"].to(torch.int64) // 16], -1).reshape(N, -1)
    if c["fmt"] == "int4":
        grp = c["group"]
        wint = (nib + 8) % 16 - 8
        for g in range(-(-K // grp)):
            a, e = g * grp, min(K, (g + 1) * grp)
            sx = _f32_quotient(x32[:, a:e].abs().amax(1), torch.tensor(7.0, device=DEV))
            live = sx > 0
            code = torch.round(_f32_quotient(x32[:, a:e], torch.where(live, sx, torch.ones_like(sx))[:, None]).double())
            code = torch.where(live[:, None], code.clamp(-7, 7), torch.zeros_like(code))
            y += (sx.double()[:, None] * code) @ (wint[:, a:e].double() * st["w_scales"][g, :N].double()[:, None]).t()
    else:
        grid = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=DEV) / 2
        gx = _f32_quotient(x32.abs().max(), torch.tensor(2688.0, device=DEV))
        byte = st["w_sf"].to(torch.int64)
        KC = -(-K // 64)
        ex, ma = byte // 8 % 16, byte % 8
        val = torch.where(ex > 0, (8 + ma).double() * torch.exp2((ex - 10).double()), ma.double() * 2.0 ** -9)
        val = val.view(-1, KC, 32, 4, 4)
        wv = torch.where(nib >= 8, -grid[nib % 8], grid[nib % 8])
        for blk in range(-(-K // 16)):
            a, e = 16 * blk, min(K, 16 * blk + 16)
            xb = x32[:, a:e]
            b8 = _f32_quotient(xb.abs().amax(1), (6 * gx.double()).float()).to(torch.float8_e4m3fn).float()
            st32 = (b8.double() * gx.double()).float()
            v = _f32_quotient(xb.abs(), torch.where(st32 > 0, st32, torch.ones_like(st32))[:, None]).double()
            d = (v[..., None] - grid).abs()
            near = d.amin(-1, keepdim=True)
            cand = d <= near  # one code, or two at a tie: the even one
            even = torch.arange(8, device=DEV) % 2 == 0
            two = cand.sum(-1, keepdim=True) > 1
            idx = torch.where(two, cand & even, cand).to(torch.int64).argmax(-1)
            code = torch.where(st32[:, None] > 0, grid[idx], torch.zeros_like(v)) * torch.where(xb < 0, -1.0, 1.0).double()
            i = torch.arange(N, device=DEV)
            bw = val[i // 128, blk // 4, i % 32, i % 128 // 32, blk % 4]
            y += (code * b8.double()[:, None]) @ (wv[:, a:e] * bw[:, None]).t()
        y *= gx.double() * st["w_gs"][0].double()
    if c["r"]:
        y += torch.einsum("mk,kr,rn->mn", x, st["L1"].double(), st["L2"].double())
    if c["bias"]:
        y += st["bias"].double()[None]
    if c["act"] == "relu":
        y = y.clamp_min(0)
    elif c["act"] == "silu":
        y = y * torch.special.expit(y)
    elif c["act"] == "gelu_tanh":
        y = y * torch.special.expit(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
    elif c["act"] == "gelu_erf":
        y = y * torch.special.ndtr(y)
    if c["mul"] == "full":
        y *= st["mul"].double()
    elif c["mul"] == "sample":
        y *= st["mul"].double()[torch.arange(M, device=DEV) // st["mul_rows"]]
    if c["residual"]:
        y += st["residual"].double()
    return y


def _exact_turn(x, turn, interleaved, scale):
    """Rotation as multiplication by a unit complex number, in 64 bits."""
    P = turn.shape[1]
    x = x.double()
    d = x[..., :2 * P]
    z = torch.view_as_complex(d.unflatten(-1, (P, 2)).contiguous()) if interleaved else torch.complex(d[..., :P], d[..., P:])
    z = z * torch.polar(torch.full_like(turn, scale), turn)[:, None]
    out = x.clone()
    out[..., :2 * P] = torch.view_as_real(z).flatten(-2) if interleaved else torch.cat((z.real, z.imag), -1)
    return out


def _exact_rope(c, seed):
    st = prepare(c, seed)
    row = torch.arange(c["tokens"], device=DEV) % c["pos_rows"]
    turn = torch.stack([st["pos"][row, a].double() * f for a, f in zip(st["axes"], st["freqs"].double())], 1)
    return _exact_turn(st["x"], -turn if c["transpose"] else turn, c["interleaved"], c["scale"])


def _exact_append(c, seed):
    st = prepare(c, seed)
    lens = st["lens"].tolist()
    cu = list(range(c["seqs"] + 1)) if st["cu"] is None else st["cu"].tolist()
    at = torch.cat([torch.arange(a, a + e - b) for a, b, e in zip(lens, cu, cu[1:])]).to(DEV)
    where = torch.cat([st["table"][i][(a + torch.arange(e - b, device=DEV)) // c["page"]] * c["page"]
                       + (a + torch.arange(e - b, device=DEV)) % c["page"]
                       for i, (a, b, e) in enumerate(zip(lens, cu, cu[1:]))]).long()
    n = st["real"]
    turn = at.double()[:, None] * st["freqs"].double()[None]
    turned = lambda x: _exact_turn(x, turn, c["interleaved"], 1.0) if c["rotate"] else x.double()  # noqa: E731
    res = {"q": st["q_out"].double()}
    res["q"][:n] = turned(st["q"][:n])
    for name, x in (("k", turned(st["k"][:n])), ("v", st["v"][:n].double())):
        cache = st[name + "_cache"]
        flat = cache.double().reshape(-1, c["kv"], c["dim"])
        scale = st[name + "_scale"]
        flat[where] = x if scale is None else (x / scale.double()[:, None]).clamp(-448, 448)
        res[name + "_cache"] = flat.view(cache.shape)
    return res


def exact(case, seed):
    return {"linear": _exact_linear, "rope": _exact_rope, "append": _exact_append}[case["op"]](dict(case), int(seed))
