"""Cases and plain forms of the operators around and inside the MoE layer:

  residual_norm            r = residual_scale x + branch_scale gate * dropout(rmsnorm(y) w_post)
                           n = rmsnorm(r) w_next                 (what joins two blocks)
  residual_norm_backward   its gradients: dx, dy, dw_post, dgate, dw_next
  dropout                  counter-based dropout, the mask recomputed from (seed, offset, row, column)
  mx_quantize              e2m1 values under one e8m0 scale per 32, and back
  mx_gemm                  activations quantised, then the grouped product with 4-bit weights
                           (optionally SwiGLU of its gate and up halves)
  mx_ffn                   the experts of the layer in 4 bits: quantise, gate_up, SwiGLU, quantise, down

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits, rounded
once; with ``own`` true it makes the calls of ``deterministic_invariant_routing_b200.moe``.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def _norm_case(kind, T, H, dtype, gate, p, post=True, nxt=True, name=None):
    c = {"kind": kind, "T": T, "H": H, "dtype": dtype, "gate": gate, "p": p, "post": post,
         "next": nxt}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token between two blocks of a decode step: pure latency
        _norm_case("residual_norm", 1, 2048, "bf16", "none", 0.0, name="norm_decode"),
        # a training batch: post-norm, learned channel gate, dropout, the next pre-norm
        _norm_case("residual_norm", 16384, 2048, "bf16", "channel", 0.1, name="norm_train"),
        # a small ragged batch kept in fp32 with a gate per token
        _norm_case("residual_norm_backward", 1021, 1000, "f32", "token", 0.25,
                   name="norm_bwd_ragged"),
        # the backward of a training batch at the wider hidden size
        _norm_case("residual_norm_backward", 8192, 4096, "bf16", "channel", 0.1,
                   name="norm_bwd_train"),
        # dropout of a small ragged fp32 activation, and of a training batch's hidden states
        {"kind": "dropout", "T": 333, "H": 128, "dtype": "f32", "p": 0.5, "name": "dropout_small"},
        {"kind": "dropout", "T": 16384, "H": 2048, "dtype": "bf16", "p": 0.1,
         "name": "dropout_train"},
        # the rows of a few decoded tokens, and the gate/up weights of 32 experts
        {"kind": "mx_quantize", "R": 61, "K": 2048, "dtype": "bf16", "name": "quant_rows"},
        {"kind": "mx_quantize", "R": 49152, "K": 2048, "dtype": "bf16", "name": "quant_weights"},
        # the down product of 64 decoded tokens (8 experts each of 128), and the gate/up product
        # of an odd prefill over 256 experts
        {"kind": "mx_gemm", "R": 512, "E": 128, "N": 2048, "K": 768, "swiglu": False,
         "name": "mx_gemm_decode"},
        {"kind": "mx_gemm", "R": 24594, "E": 256, "N": 2048, "K": 4096, "swiglu": True,
         "name": "mx_gemm_prefill"},
        # the whole expert stage for a single token, and for a full prefill batch
        {"kind": "mx_ffn", "T": 1, "H": 2048, "E": 128, "K": 8, "I": 768, "name": "mx_ffn_decode"},
        {"kind": "mx_ffn", "T": 16384, "H": 2048, "E": 128, "K": 8, "I": 768,
         "name": "mx_ffn_prefill"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["residual_norm", "residual_norm_backward", "dropout", "mx_quantize",
                       "mx_gemm", "mx_ffn"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind in ("residual_norm", "residual_norm_backward"):
        H = 8 * _log(rng, 8, 1024)
        T = _log(rng, 1, max(1, (1 << 24) // H))
        p = rng.choice([0.0, round(rng.uniform(0.01, 0.6), 3)])
        return _norm_case(kind, T, H, dtype, rng.choice(["none", "channel", "token", "full"]), p,
                          rng.random() < 0.8, rng.random() < 0.8)
    if kind == "dropout":
        H = 8 * _log(rng, 1, 1024)
        return {"kind": kind, "T": _log(rng, 1, (1 << 24) // H), "H": H, "dtype": dtype,
                "p": round(rng.uniform(0.001, 0.9), 4)}
    if kind == "mx_quantize":
        K = 32 * _log(rng, 1, 256)
        return {"kind": kind, "R": _log(rng, 1, (1 << 25) // K), "K": K, "dtype": dtype}
    if kind == "mx_gemm":
        E, N, K = _log(rng, 1, 96), 256 * _log(rng, 1, 11), 128 * _log(rng, 1, 23)
        return {"kind": kind, "R": _log(rng, 1, 24000), "E": E, "N": N, "K": K,
                "swiglu": rng.random() < 0.5}
    E = _log(rng, 8, 96)
    return {"kind": kind, "T": _log(rng, 1, 6000), "H": 128 * _log(rng, 1, 20), "E": E,
            "K": rng.randint(1, min(8, E)), "I": 128 * _log(rng, 1, 11)}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, g, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _uneven(rows, E, g):
    """Rows per expert under uneven loads (a log-normal popularity), and their offsets."""
    pop = torch.exp(0.5 * torch.randn(E, generator=g, device=DEV))
    pick = torch.multinomial(pop, rows, replacement=True, generator=g)
    sizes = torch.bincount(pick, minlength=E)
    return sizes, torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).int()


def _mx_weight(shape, g):
    """Quantised weights: codes [E, N, K/2] and the scales in tiles of 128 rows by 4 blocks,
    [E, N/128, K/128, 512] (row r of a tile at 16 (r % 32) + 4 (r / 32), its 4 blocks in order)."""
    E, N, K = shape
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(E, N, K // 32, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        w = _normal((n, N, K), g, torch.bfloat16, 0.02)
        codes[e:e + n], scales[e:e + n] = _quantize(w)
    tiled = scales.view(E, N // 128, 4, 32, K // 128, 4).permute(0, 1, 4, 3, 2, 5)
    return codes, tiled.reshape(E, N // 128, K // 128, 512).contiguous()


def prepare(case, seed):
    g, kind = _gen(seed), case["kind"]
    if kind in ("residual_norm", "residual_norm_backward"):
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        s = {"case": case, "y": _normal((T, H), g, dt, 0.5), "w_post": None, "w_next": None,
             "gate": None, "rng": torch.tensor([seed * 7919 + 1, 3], device=DEV)}
        if case["post"]:
            s["w_post"] = 1 + _normal((H,), g, torch.float32, 0.1)
        if case["next"]:
            s["w_next"] = 1 + _normal((H,), g, torch.float32, 0.1)
        shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[case["gate"]]
        if shape:
            s["gate"] = _normal(shape, g, dt if case["gate"] == "full" else torch.float32, 0.5)
        if kind == "residual_norm":
            s["x"] = _normal((T, H), g, dt)
        else:
            s["r"] = _normal((T, H), g, dt)
            s["dr"] = _normal((T, H), g, dt, 0.1)
            s["dn"] = _normal((T, H), g, dt, 0.1) if case["next"] else None
        return s
    if kind == "dropout":
        x = _normal((case["T"], case["H"]), g, DTYPES[case["dtype"]])
        return {"case": case, "x": x, "rng": torch.tensor([seed * 104729 + 5, 11], device=DEV)}
    if kind == "mx_quantize":
        x = _normal((case["R"], case["K"]), g, DTYPES[case["dtype"]])
        x *= torch.exp2(torch.randint(-6, 7, (case["R"], 1), generator=g, device=DEV).float())
        return {"case": case, "x": x}
    if kind == "mx_gemm":
        R, E, N, K = case["R"], case["E"], case["N"], case["K"]
        sizes, offsets = _uneven(R, E, g)
        codes, scales = _mx_weight((E, N, K), g)
        return {"case": case, "x": _normal((R, K), g, torch.bfloat16), "offsets": offsets,
                "sizes": sizes.tolist(), "w": (codes, scales)}
    T, H, E, K, I = (case[k] for k in ("T", "H", "E", "K", "I"))
    # the dispatch of a routed batch: K distinct experts per token, rows sorted by expert
    pop = torch.randn(T, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g,
                                                                         device=DEV)
    ids = pop.topk(K, dim=1).indices
    order = ids.reshape(-1).argsort(stable=True)
    dest = torch.empty(T * K, dtype=torch.int32, device=DEV)
    dest[order] = torch.arange(T * K, dtype=torch.int32, device=DEV)
    sizes = torch.bincount(ids.reshape(-1), minlength=E)
    offsets = torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).int()
    return {"case": case, "x": _normal((T, H), g, torch.bfloat16), "dest_row": dest.view(T, K),
            "rows": order // K, "offsets": offsets, "sizes": sizes.tolist(),
            "w13": _mx_weight((E, 2 * I, H), g), "w2": _mx_weight((E, H, I), g)}


# ------------------------------------------------------------------ plain forms

def _philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 on int64 tensors holding 32-bit words."""
    m = 0xFFFFFFFF
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & m) ^ c1 ^ k0, p1 & m, ((p0 >> 32) & m) ^ c3 ^ k1, p0 & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    return c0, c1, c2, c3


def _keep(T, H, p, rng):
    """(keep [T, H], 1 / probability to keep): 16 bits per element, eight elements per counter
    (column / 8, row, offset), the key the seed."""
    m = 0xFFFFFFFF
    threshold = math.floor(p * 65536 + 0.5)
    col = torch.arange(H // 8, device=DEV).expand(T, -1)
    row = torch.arange(T, device=DEV)[:, None].expand(-1, H // 8)
    words = _philox(col, row, (rng[1] & m).expand_as(col), ((rng[1] >> 32) & m).expand_as(col),
                    rng[0] & m, (rng[0] >> 32) & m)
    u = torch.stack([w for v in words for w in (v & 0xFFFF, v >> 16)], dim=-1).view(T, H)
    return u >= threshold, 65536 / (65536 - threshold)


def _rms(v):
    return torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _residual_norm(s):
    c = s["case"]
    dt = s["x"].dtype
    b = s["y"].float()
    if c["post"]:
        b = b * _rms(b) * s["w_post"]
    if c["p"]:
        keep, inv = _keep(c["T"], c["H"], c["p"], s["rng"])
        b = torch.where(keep, b * inv, 0.0)
    if s["gate"] is not None:
        b = b * s["gate"].float()
    r = (0.8 * s["x"].float() + 0.6 * b).to(dt)
    if not c["next"]:
        return {"r": r}
    f = r.float()
    return {"r": r, "n": (f * _rms(f) * s["w_next"]).to(dt)}


def _norm_grad(v, w, d):
    """Gradients (dv, dw) of rmsnorm(v) * w for the output gradient d."""
    s = _rms(v)
    hat, dw = v * s, d * w
    return s * (dw - hat * (dw * hat).mean(-1, keepdim=True)), (d * hat).sum(0)


def _residual_norm_backward(s):
    c, out = s["case"], {}
    dt, gate = s["y"].dtype, s["gate"]
    d = s["dr"].float()
    if c["next"]:
        dv, out["dw_next"] = _norm_grad(s["r"].float(), s["w_next"], s["dn"].float())
        d = d + dv
    out["dx"] = (0.8 * d).to(dt)
    d = 0.6 * d
    y = s["y"].float()
    z = y * _rms(y) * s["w_post"] if c["post"] else y
    if c["p"]:
        keep, inv = _keep(c["T"], c["H"], c["p"], s["rng"])
        z = torch.where(keep, z * inv, 0.0)
    if gate is not None:
        dg = d * z
        out["dgate"] = {"channel": lambda: dg.sum(0), "token": lambda: dg.sum(1, keepdim=True),
                        "full": lambda: dg.to(dt)}[c["gate"]]()
        d = d * gate.float()
    if c["p"]:
        d = torch.where(keep, d * inv, 0.0)
    if c["post"]:
        d, out["dw_post"] = _norm_grad(y, s["w_post"], d)
    out["dy"] = d.to(dt)
    return out


def _pow2(e):
    """2^e, exactly (a power function may be off in its last place)."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _quantize(x):
    """e2m1 codes (two per byte, even column in the low nibble) and e8m0 scales, one per 32
    columns: the scale 2^(floor(log2 amax) - 2), values to nearest even, saturated at 6."""
    v = x.float().unflatten(-1, (-1, 32))
    e = (torch.frexp(v.abs().amax(-1)).exponent - 3).clamp(-127, 127)
    a = v.abs() * _pow2(-e)[..., None]
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) +
            (a >= 3.5) + (a > 5.0)) | (v < 0).to(torch.uint8) << 3
    code = code.flatten(-2).unflatten(-1, (-1, 2))
    return code[..., 0] | code[..., 1] << 4, (e + 127).to(torch.uint8)


def _values(codes, scales, dtype=torch.float32):
    """The values that codes [..., K/2] and scales [..., K/32] stand for."""
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=dtype, device=DEV)
    e2m1 = torch.cat([e2m1, -e2m1])
    v = torch.stack([e2m1[(codes & 15).int()], e2m1[(codes >> 4).int()]], -1).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * _pow2(scales.int() - 127)[..., None]).flatten(-2)


def _weights(w, experts, dtype=torch.float32):
    """The values of these experts' weights, [experts, N, K]."""
    codes, tiled = (v[experts] for v in w)
    n, N, K2 = codes.shape
    scales = tiled.view(n, N // 128, K2 // 64, 32, 4, 4).permute(0, 1, 4, 3, 2, 5)
    return _values(codes, scales.reshape(n, N, K2 // 16), dtype)


def _product(a, w, sizes, swiglu):
    """Rows grouped by expert against that expert's weights; with swiglu, silu(gate) * up."""
    experts = [e for e, n in enumerate(sizes) if n]
    v = torch.cat([p @ q.T for p, q in zip(a.split([sizes[e] for e in experts]),
                                           _weights(w, experts))])
    if swiglu:
        gate, up = v.chunk(2, dim=1)
        v = gate * torch.sigmoid(gate) * up
    return v


def _plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "residual_norm":
        return _residual_norm(s)
    if kind == "residual_norm_backward":
        return _residual_norm_backward(s)
    if kind == "dropout":
        keep, inv = _keep(c["T"], c["H"], c["p"], s["rng"])
        return torch.where(keep, s["x"].float() * inv, 0.0).to(s["x"].dtype)
    if kind == "mx_quantize":
        return _values(*_quantize(s["x"])).to(torch.bfloat16)
    if kind == "mx_gemm":
        a = _values(*_quantize(s["x"]))
        return _product(a, s["w"], s["sizes"], c["swiglu"]).to(torch.bfloat16)
    a = _values(*_quantize(s["x"]))[s["rows"]]
    h = _product(a, s["w13"], s["sizes"], True).to(torch.bfloat16)
    return _product(_values(*_quantize(h)), s["w2"], s["sizes"], False).to(torch.bfloat16)


# ------------------------------------------------------------------ one pass

def _own(s):
    from deterministic_invariant_routing_b200 import moe
    c = s["case"]
    kind = c["kind"]
    if kind == "residual_norm":
        r, n = moe.residual_norm(s["x"], s["y"], w_post=s["w_post"], gate=s["gate"],
                                 w_next=s["w_next"], eps=EPS, residual_scale=0.8,
                                 branch_scale=0.6, p=c["p"], rng=s["rng"])
        return {"r": r, "n": n} if c["next"] else {"r": r}
    if kind == "residual_norm_backward":
        return moe.residual_norm_backward(s["r"], s["y"], dr=s["dr"], dn=s["dn"],
                                          w_post=s["w_post"], gate=s["gate"], w_next=s["w_next"],
                                          eps=EPS, residual_scale=0.8, branch_scale=0.6,
                                          p=c["p"], rng=s["rng"])
    if kind == "dropout":
        return moe.dropout(s["x"], c["p"], s["rng"])
    if kind == "mx_quantize":
        return moe.mx_dequantize(*moe.mx_quantize(s["x"]))
    if kind == "mx_gemm":
        codes, scales = moe.mx_quantize(s["x"])
        return moe.mx_grouped_gemm(codes, scales, s["offsets"], *s["w"], swiglu=c["swiglu"],
                                   check=False)
    cfg = moe.Config(T=c["T"], H=c["H"], E=c["E"], K=c["K"], I=c["I"])
    return moe.mx_grouped_ffn(cfg, s["x"], s["dest_row"], s["offsets"], s["w13"], s["w2"],
                              check=False)[0]


def run(state):
    return _own(state) if own else _plain(state)


def _touched(rows, E):
    """Experts that `rows` picks among E reach, at most."""
    return min(rows, E)


def work(case):
    kind = case["kind"]
    if kind in ("residual_norm", "residual_norm_backward"):
        T, H = case["T"], case["H"]
        b = 4 if case["dtype"] == "f32" else 2
        full = case["gate"] == "full"
        per_h = 4 * (int(case["post"]) + int(case["next"]) + int(case["gate"] == "channel"))
        if kind == "residual_norm":  # x, y (and a full gate) in, r and n out
            passes = 3 + int(case["next"]) + int(full)
            return {"bytes": T * H * b * passes + H * per_h, "flops": 14 * T * H}
        # y, dr (and r, dn, a full gate) in, dx, dy (and its gradient) out
        passes = 4 + 2 * int(case["next"]) + 2 * int(full)
        return {"bytes": T * H * b * passes + 2 * H * per_h, "flops": 30 * T * H}
    if kind == "dropout":
        b = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * b * case["T"] * case["H"], "flops": 2 * case["T"] * case["H"]}
    if kind == "mx_quantize":
        b = 4 if case["dtype"] == "f32" else 2
        n = case["R"] * case["K"]
        return {"bytes": n * (b + 2), "flops": 4 * n}
    if kind == "mx_gemm":
        R, E, N, K = (case[k] for k in ("R", "E", "N", "K"))
        out = N // 2 if case["swiglu"] else N
        return {"bytes": R * K * 2 + _touched(R, E) * N * K * 17 // 32 + R * out * 2,
                "flops": 2 * R * N * K}
    T, H, E, K, I = (case[k] for k in ("T", "H", "E", "K", "I"))
    return {"bytes": T * H * 2 + _touched(T * K, E) * 3 * H * I * 17 // 32 + T * K * H * 2,
            "flops": 6 * T * K * H * I}


# ------------------------------------------------------------------ 64 bits

def _keep64(c, rng):
    """The mask from Python's own integers for the key, the counters in int64 tensors split into
    16-bit halves (no product over 48 bits)."""
    T, H = c["T"], c["H"]
    seed, offset = (v & 0xFFFFFFFFFFFFFFFF for v in rng.tolist())

    def mulhilo(a, b):  # (high, low) words of a * b, b a 32-bit constant
        lo, hi = (a & 0xFFFF) * b, (a >> 16) * b
        low = lo + ((hi & 0xFFFF) << 16)
        return (hi >> 16) + (low >> 32), low & 0xFFFFFFFF

    x = [torch.arange(H // 8, device=DEV)[None].repeat(T, 1),
         torch.arange(T, device=DEV)[:, None].repeat(1, H // 8),
         torch.full((T, H // 8), offset & 0xFFFFFFFF, device=DEV),
         torch.full((T, H // 8), offset >> 32, device=DEV)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for i in range(10):
        h0, l0 = mulhilo(x[0], 0xD2511F53)
        h1, l1 = mulhilo(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    out = torch.empty(T, H // 8, 8, dtype=torch.int64, device=DEV)
    for i, w in enumerate(x):
        out[..., 2 * i], out[..., 2 * i + 1] = w % 65536, w // 65536
    drop = math.floor(c["p"] * 65536 + 0.5)
    return (out.view(T, H) >= drop).double() * (65536 / (65536 - drop))


def _exact_norm(case, s):
    c = case
    y = s["y"].double()
    T, H = y.shape
    mask = _keep64(c, s["rng"]) if c["p"] else torch.ones_like(y)
    wp = s["w_post"].double() if c["post"] else None
    gate = s["gate"].double() if s["gate"] is not None else torch.ones(1, 1, device=DEV,
                                                                       dtype=torch.float64)
    inv_y = ((y.square().sum(1) / H + EPS) ** -0.5)[:, None]
    z = (y * inv_y * wp if c["post"] else y) * mask
    if c["kind"] == "residual_norm":
        r = 0.8 * s["x"].double() + 0.6 * gate * z
        out = {"r": r}
        if c["next"]:  # by definition of the stored, rounded r
            q = r.to(s["x"].dtype).double()
            out["n"] = q / (q.square().sum(1) / H + EPS).sqrt()[:, None] * s["w_next"].double()
        return out
    total, out = s["dr"].double(), {}
    if c["next"]:
        r, dn, w = s["r"].double(), s["dn"].double(), s["w_next"].double()
        i = ((r.square().sum(1) / H + EPS) ** -0.5)[:, None]
        out["dw_next"] = torch.einsum("th,th->h", dn, r * i)
        total = total + i * dn * w - r * i ** 3 * ((dn * w * r).sum(1) / H)[:, None]
    out["dx"] = 0.8 * total
    branch = 0.6 * total
    if c["gate"] == "channel":
        out["dgate"] = torch.einsum("th,th->h", branch, z)
    elif c["gate"] == "token":
        out["dgate"] = torch.einsum("th,th->t", branch, z)[:, None]
    elif c["gate"] == "full":
        out["dgate"] = branch * z
    d = branch * gate * mask
    if c["post"]:
        out["dw_post"] = torch.einsum("th,th->h", d, y * inv_y)
        d = inv_y * d * wp - y * inv_y ** 3 * ((d * wp * y).sum(1) / H)[:, None]
    out["dy"] = d
    return out


def _fake64(x):
    """x in 64 bits after the 4-bit format: each block of 32 to the nearest of the scaled e2m1
    values (even codes win ties), beyond the largest to the largest."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    mid = (grid[1:] + grid[:-1]) / 2
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -125)
    step = (((top.view(torch.int64) >> 52) - 2) << 52).view(torch.float64)  # its exponent, less 2
    a = b.abs() / step
    up, down = torch.bucketize(a, mid, right=True), torch.bucketize(a, mid)
    at = torch.where((up != down) & (up % 2 == 1), down, up)  # on a border: the even code
    return (torch.sign(b) * grid[at] * step).reshape(x.shape)


def _exact_product(a, w, sizes, swiglu):
    parts, at = [], 0
    for e, n in enumerate(sizes):
        v = torch.matmul(a[at:at + n], _weights(w, [e], torch.float64)[0].T)
        at += n
        if swiglu:
            g, u = v.chunk(2, dim=1)
            v = g / (1 + torch.exp(-g)) * u
        parts.append(v)
    return torch.cat(parts)


def exact(case, seed):
    s, kind = prepare(case, seed), case["kind"]
    if kind in ("residual_norm", "residual_norm_backward"):
        return _exact_norm(case, s)
    if kind == "dropout":
        return s["x"].double() * _keep64(case, s["rng"])
    if kind == "mx_quantize":
        return _fake64(s["x"])
    if kind == "mx_gemm":
        return _exact_product(_fake64(s["x"]), s["w"], s["sizes"], case["swiglu"])
    h = _exact_product(_fake64(s["x"])[s["rows"]], s["w13"], s["sizes"], True)
    return _exact_product(_fake64(h.to(torch.bfloat16)), s["w2"], s["sizes"], False)
