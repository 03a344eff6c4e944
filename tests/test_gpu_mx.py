"""The 4-bit experts on the GPU: format, products, the expert stage and the layer.

Quantisation is compared code by code. Products: every product of two e2m1 values and powers of
two is exact in fp32, the tensor core adds K of them (K roundings of at most 2^-24 of the sum of
the magnitudes), then one rounding to bf16: 8 significant bits, a step of 2^-7 of the value at
a power of two, so half a step is at most 2^-8 of it (torch.finfo(bfloat16).eps / 2).
SwiGLU: the errors of gate and up carried to first order, and 2^-17 of the value for the
hardware exponential (2 ulp, and its argument's rounding, |g| 2^-24 with |g| below 60). The
expert stage is compared bit by bit with the calls it replaces."""
import pytest
import torch

import mx_ref as M
from deterministic_invariant_routing_b200 import _native as N
from deterministic_invariant_routing_b200 import moe, synthetic
from helpers import DEV, bits

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rows_like(shape, seed, dt=torch.bfloat16):
    g = gen(seed)
    x = torch.randn(shape, generator=g, device=DEV)
    return (x * torch.exp2(torch.randint(-8, 9, (*shape[:-1], 1), generator=g, device=DEV))).to(dt)


def eq(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ------------------------------------------------------------------ format

@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("R,K", [(1, 32), (3, 96), (61, 2048), (257, 1056), (1025, 128)])
def test_quantize_codes_and_values(dt, R, K):
    x = rows_like((R, K), R + K, TYPES[dt])
    x[0] = 0
    if R > 2:  # every tie of the grid, each sign, on the scale 1
        t = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
        x[2, :16] = torch.cat([t, -t]).to(TYPES[dt])
        x[2, 16:32] = 0
        x[1, :32] = torch.finfo(TYPES[dt]).smallest_normal
        x[1, 0] = torch.finfo(TYPES[dt]).max
    codes, scales = moe.mx_quantize(x, tiled=False)
    ref, rs = M.quantize64(x)
    assert torch.equal(scales, rs)
    assert torch.equal(M.unpack(codes), ref)
    c2, tiles = moe.mx_quantize(x)
    assert torch.equal(c2, codes)
    pad = torch.zeros(-(-R // 128) * 128, -(-K // 128) * 4, dtype=torch.uint8, device=DEV)
    pad[:R, :K // 32] = rs
    assert torch.equal(M.untile(tiles), pad)  # the padding's scales are 0
    for out in TYPES.values():
        want = M.values64(codes, scales).to(out)
        assert torch.equal(moe.mx_dequantize(codes, scales, out), want)
        assert torch.equal(moe.mx_dequantize(codes, tiles, out), want)


def test_quantize_subnormals_and_extremes():
    """fp32 blocks at the ends of the range: the scale clamps at 2^-127, subnormals round."""
    x = torch.zeros(6, 32, device=DEV)
    x[0, 1], x[1, 2], x[2, 3] = 2.0 ** -149, 2.0 ** -128, 1.5 * 2.0 ** -126
    x[3], x[4, 0], x[5, 5] = torch.finfo(torch.float32).max, 2.0 ** -125, 5 * 2.0 ** -127
    codes, scales = moe.mx_quantize(x, tiled=False)
    ref, rs = M.quantize64(x)
    assert torch.equal(scales, rs) and torch.equal(M.unpack(codes), ref)


def test_non_finite_blocks():
    x = torch.ones(4, 128, device=DEV)
    x[0, 5], x[1, 40], x[2, 127] = float("nan"), float("inf"), float("-inf")
    codes, scales = moe.mx_quantize(x, tiled=False)
    want = torch.full((4, 4), 125, dtype=torch.uint8)
    want[0, 0] = want[1, 1] = want[2, 3] = 255
    assert torch.equal(scales.cpu(), want)
    v = moe.mx_dequantize(codes, scales, torch.float32)
    nan = (want == 255).repeat_interleave(32, 1).to(DEV)
    assert torch.equal(v.isnan(), nan) and torch.equal(v[~nan], x[~nan])
    assert not M.unpack(codes)[nan].any()


@pytest.mark.parametrize("shape", [(128, 128), (3, 256, 384), (2, 128, 2048)])
def test_weights_keep_their_scales_in_tiles(shape):
    w = rows_like(shape, 7)
    codes, tiled = moe.mx_weight(w)
    ref, rs = M.quantize64(w)
    assert torch.equal(M.unpack(codes), ref) and torch.equal(M.untile(tiled), rs)
    c2, s2 = moe.mx_quantize(w.view(-1, shape[-1]), tiled=False)
    assert torch.equal(c2.view_as(codes), codes) and torch.equal(s2.view_as(rs), rs)


# ------------------------------------------------------------------ products

def make_product(sizes, N_, K, seed=0, start=0, extra=0):
    E, R = len(sizes), start + sum(sizes) + extra
    x = rows_like((R, K), seed)
    w = rows_like((E, N_, K), seed + 1) * 0.02
    off = [start]
    for n in sizes:
        off.append(off[-1] + n)
    return x, w, off


def check_product(out, x, w, off, swiglu, K):
    a = M.values64(*moe.mx_quantize(x, tiled=False))
    wc, ws = moe.mx_weight(w)
    ref, mag = M.product64(a, M.values64(wc, M.untile(ws)), off, swiglu)
    tol = 2.0 ** -8 * ref.abs() + K * 2.0 ** -24 * mag + (2.0 ** -17 * ref.abs() if swiglu else 0)
    s = slice(off[0], off[-1])
    err = (out[s].double() - ref[s]).abs()
    worst = (err / (tol[s] + 1e-38)).max().item() if err.numel() else 0.0
    assert worst <= 1.0, worst


PRODUCTS = [([1], 128, 128), ([0, 1, 0], 256, 128), ([5, 0, 31, 33], 256, 384), ([128], 256, 256),
            ([129, 127], 384, 512), ([256, 257, 1], 256, 768), ([700], 512, 2048),
            ([3] * 40, 256, 256), ([0, 0, 900, 0], 768, 128), ([64, 0, 511, 2, 1], 1280, 1152),
            ([40, 9], 256, 4096), ([20] * 130, 128, 128)]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("case", range(len(PRODUCTS)))
def test_grouped_product(case, swiglu):
    sizes, n, K = PRODUCTS[case]
    if swiglu and n % 256:
        n += 128
    x, w, off = make_product(sizes, n, K, seed=case)
    out = moe.mx_grouped_gemm(*moe.mx_quantize(x), torch.tensor(off, dtype=torch.int32, device=DEV),
                              *moe.mx_weight(w), swiglu=swiglu)
    check_product(out, x, w, off, swiglu, K)


@pytest.mark.parametrize("swiglu", [False, True])
def test_rows_outside_the_groups_are_left(swiglu):
    x, w, off = make_product([37, 0, 300], 256, 256, start=11, extra=45)
    out = torch.full((x.shape[0], 128 if swiglu else 256), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.mx_grouped_gemm(*moe.mx_quantize(x), torch.tensor(off, dtype=torch.int32, device=DEV),
                        *moe.mx_weight(w), swiglu=swiglu, out=out)
    assert (out[:11] == 7).all() and (out[off[-1]:] == 7).all()
    check_product(out, x, w, off, swiglu, 256)


@pytest.mark.parametrize("start,n", [(0, 31), (1, 31), (0, 32), (31, 65), (31, 66), (30, 67),
                                     (62, 66), (0, 97), (0, 98), (31, 97), (127, 1), (127, 2)])
def test_few_rows_at_every_place_of_a_tile(start, n):
    """Calls of so few rows that whole boxes and store tiles just do or do not occur."""
    x, w, off = make_product([n], 256, 384, seed=n, start=start)
    for swiglu in (False, True):
        out = moe.mx_grouped_gemm(*moe.mx_quantize(x),
                                  torch.tensor(off, dtype=torch.int32, device=DEV),
                                  *moe.mx_weight(w), swiglu=swiglu)
        check_product(out, x, w, off, swiglu, 384)


def test_many_tiles_a_cluster():
    """More tiles than clusters take at once, uneven groups: every role keeps its phases."""
    g = torch.randperm(64, generator=torch.Generator().manual_seed(1)).tolist()
    sizes = [17 * v for v in g]
    x, w, off = make_product(sizes, 768, 640)
    out = moe.mx_grouped_gemm(*moe.mx_quantize(x), torch.tensor(off, dtype=torch.int32, device=DEV),
                              *moe.mx_weight(w), swiglu=True)
    check_product(out, x, w, off, True, 640)


def test_a_row_keeps_its_bits_anywhere():
    """The same rows alone, in other groups' company, at other places of a tile."""
    K, n = 896, 512
    w = moe.mx_weight(rows_like((3, n, K), 5) * 0.02)
    x = rows_like((600, K), 6)

    def run(rows, off, glu):
        i = torch.tensor(rows, device=DEV)
        return moe.mx_grouped_gemm(*moe.mx_quantize(x[i]),
                                   torch.tensor(off, dtype=torch.int32, device=DEV), *w,
                                   swiglu=glu)

    for glu in (False, True):
        full = run(list(range(600)), [0, 100, 500, 600], glu)
        part = run(list(range(90, 100)) + list(range(301, 500)) + [599], [0, 10, 209, 210], glu)
        assert eq(part, torch.cat([full[90:100], full[301:500], full[599:]]))
        one = run([444], [0, 0, 1, 1], glu)
        assert eq(one, full[444:445])
        assert eq(run(list(range(600)), [0, 100, 500, 600], glu), full)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("sizes", [[64] * 4, [65, 64, 64, 64], [3, 250, 0, 3], [0, 300, 1, 1],
                                   [1] * 150, [130, 5] * 30])
def test_few_and_many_rows_a_group(sizes, glu):
    """Up to 64 rows a group on average, and above, where the row tiles change."""
    x, w, off = make_product(sizes, 384 + 128 * glu, 384, seed=len(sizes),
                             extra=64 * (sizes[0] == 0))
    out = moe.mx_grouped_gemm(*moe.mx_quantize(x),
                              torch.tensor(off, dtype=torch.int32, device=DEV),
                              *moe.mx_weight(w), swiglu=glu)
    check_product(out[:off[-1]], x[:off[-1]], w, off, glu, 384)
    lone = sum(sizes[:2]) - 1  # the second group's last row, computed by itself
    one = moe.mx_grouped_gemm(*moe.mx_quantize(x[lone:lone + 1]),
                              torch.tensor([0, 0, 1] + [1] * (len(sizes) - 2),
                                           dtype=torch.int32, device=DEV),
                              *moe.mx_weight(w), swiglu=glu)
    assert eq(one, out[lone:lone + 1])


@pytest.mark.parametrize("groups", [320, 321, 1024])
def test_many_groups(groups):
    """More groups than a block has threads, empty ones and a decreasing offset among them."""
    sizes = [(7 * i) % 5 if i % 3 else 0 for i in range(groups)]
    sizes[-1], sizes[200] = 150, 140
    x, w, off = make_product(sizes, 128, 128, seed=groups)
    q, wq = moe.mx_quantize(x), moe.mx_weight(w)
    out = moe.mx_grouped_gemm(*q, torch.tensor(off, dtype=torch.int32, device=DEV), *wq)
    check_product(out, x, w, off, False, 128)
    off[300] -= 1000
    st = moe.new_status(DEV)
    moe.mx_grouped_gemm(*q, torch.tensor(off, dtype=torch.int32, device=DEV), *wq, status=st,
                        check=False)
    assert st[N.MOE_ST_BAD_ROWS] > 0


def test_nan_blocks_reach_their_results_alone():
    x, w, off = make_product([200, 100], 256, 512, seed=3)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    clean = moe.mx_grouped_gemm(*moe.mx_quantize(x), offs, *moe.mx_weight(w))
    xb, wb = x.clone(), w.clone()
    xb[17, 333] = float("nan")
    wb[1, 40, 500] = float("inf")
    out = moe.mx_grouped_gemm(*moe.mx_quantize(xb), offs, *moe.mx_weight(wb))
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[17] = True
    nan[200:, 40] = True
    assert torch.equal(out.isnan(), nan) and torch.equal(out[~nan], clean[~nan])


def test_bad_offsets_and_rows_are_counted():
    """Offsets past the rows, negative or decreasing are clamped by the kernel and counted;
    destinations past T*K likewise; the next call is clean."""
    x, w, off = make_product([10, 20, 30], 256, 128)
    q, wq = moe.mx_quantize(x), moe.mx_weight(w)
    for bad in ([0, 10, 30, 61], [-1, 10, 30, 60], [0, 40, 30, 60], [0, 10, 30, 2 ** 31 - 1]):
        st = moe.new_status(DEV)
        moe.mx_grouped_gemm(*q, torch.tensor(bad, dtype=torch.int32, device=DEV), *wq, status=st,
                            check=False)
        assert st[N.MOE_ST_BAD_ROWS] > 0
        with pytest.raises(moe.StatusError, match="bad_rows"):
            moe.mx_grouped_gemm(*q, torch.tensor(bad, dtype=torch.int32, device=DEV), *wq)
    out = moe.mx_grouped_gemm(*q, torch.tensor(off, dtype=torch.int32, device=DEV), *wq)
    check_product(out, x, w, off, False, 128)
    cfg = moe.Config(T=4, H=128, E=2, K=1, I=128)
    dest = torch.tensor([[0], [1], [2], [4]], dtype=torch.int32, device=DEV)
    o = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    w13, w2 = moe.mx_weight(rows_like((2, 256, 128), 1)), moe.mx_weight(rows_like((2, 128, 128), 2))
    with pytest.raises(moe.StatusError, match="bad_rows"):
        moe.mx_grouped_ffn(cfg, rows_like((4, 128), 3), dest, o, w13, w2)


def test_no_rows():
    x, w, off = make_product([0, 0], 256, 128)
    out = moe.mx_grouped_gemm(*moe.mx_quantize(x), torch.zeros(3, dtype=torch.int32, device=DEV),
                              *moe.mx_weight(w))
    assert out.shape == (0, 256)
    x = rows_like((5, 128), 1)
    out = torch.full((5, 256), 3.0, dtype=torch.bfloat16, device=DEV)
    moe.mx_grouped_gemm(*moe.mx_quantize(x), torch.zeros(3, dtype=torch.int32, device=DEV),
                        *moe.mx_weight(w), out=out)
    assert (out == 3).all()
    assert moe.mx_dequantize(*moe.mx_quantize(x[:0])).shape == (0, 128)
    st = torch.ones(N.MOE_STATUS_WORDS, dtype=torch.int32, device=DEV)
    moe.mx_grouped_gemm(*moe.mx_quantize(x[:0]), torch.zeros(3, dtype=torch.int32, device=DEV),
                        *moe.mx_weight(w), status=st)  # what an earlier call left is cleared
    cfg = moe.Config(T=0, H=128, E=2, K=1, I=128)
    w2 = moe.mx_weight(w[:, :128].contiguous())
    y, _ = moe.mx_grouped_ffn(cfg, x[:0], torch.zeros(0, 1, dtype=torch.int32, device=DEV),
                              torch.zeros(3, dtype=torch.int32, device=DEV), moe.mx_weight(w), w2,
                              status=st.fill_(1))
    assert y.shape == (0, 128)


# ------------------------------------------------------------------ the expert stage, the layer

def layer(name, T, mask=False, **over):
    s, d = synthetic.make_layer(name, T=T, device=DEV, **over)
    cfg = moe.Config.of(s)
    q = {k: moe.mx_weight(d[k]) for k in ("w13", "w2", "w13_s", "w2_s") if d.get(k) is not None}
    m = None
    if mask:
        m = torch.ones(T, dtype=torch.uint8, device=DEV)
        m[T // 3:T // 2] = 0
    return cfg, d, q, m


def staged(cfg, d, q, dest, offsets):
    """The stage by its public parts: quantise, gather, product, quantise, product."""
    n = int(offsets[-1])
    tok = torch.empty(n, dtype=torch.long, device=DEV)
    t, j = (dest >= 0).nonzero(as_tuple=True)
    tok[dest[t, j].long()] = t
    h = moe.mx_grouped_gemm(*moe.mx_quantize(d["x"][tok]), offsets, *q["w13"], swiglu=True)
    y = moe.mx_grouped_gemm(*moe.mx_quantize(h), offsets, *q["w2"])
    if not cfg.I_shared:
        return y, None
    one = torch.tensor([0, cfg.T], dtype=torch.int32, device=DEV)
    hs = moe.mx_grouped_gemm(*moe.mx_quantize(d["x"]), one, q["w13_s"][0][None], q["w13_s"][1][None], swiglu=True)
    return y, moe.mx_grouped_gemm(*moe.mx_quantize(hs), one, q["w2_s"][0][None], q["w2_s"][1][None])


@pytest.mark.parametrize("name,T,mask", [("tiny", 64, False), ("tiny", 1, False), ("tiny", 37, True),
                                         ("qwen3_30b_a3b", 1, False), ("qwen3_30b_a3b", 300, True),
                                         ("dsv_sigmoid", 65, True), ("dspark", 130, False)])
def test_stage_and_layer_equal_their_parts(name, T, mask):
    cfg, d, q, m = layer(name, T, mask)
    kw = dict(logit_bias=d["logit_bias"], sel_bias=d["sel_bias"])
    logits, ids, tw = moe.route(cfg, x=d["x"], w_router=d["w_router"], token_mask=m, **kw)
    offsets, _, dest, _ = moe.permute(cfg, ids, want_x_perm=False)
    y, ys = moe.mx_grouped_ffn(cfg, d["x"], dest, offsets, **q)
    y2, ys2 = staged(cfg, d, q, dest, offsets)
    assert eq(y[:y2.shape[0]], y2) and (ys is None or eq(ys, ys2))
    out = moe.combine(cfg, y, tw, dest, y_shared=ys, token_mask=m)
    got, b = moe.mx_forward(cfg, d["x"], d["w_router"], **q, token_mask=m, keep=True, **kw)
    assert eq(got, out) and eq(b["topk_ids"], ids) and eq(b["logits"], logits)
    assert eq(b["topk_w"], tw) and eq(b["offsets"], offsets)


def test_layer_near_the_64_bit_layer_of_its_values():
    """Against the expert formula in double on the dequantised weights and inputs, h quantised
    as defined: rows differ by bf16 roundings and by the few elements of h that fall on the
    other side of a border, so each row's largest error stays below 2^-5 of its largest value
    and the mean below 2^-8."""
    cfg, d, q, _ = layer("qwen3_30b_a3b", 48)
    logits, ids, tw = moe.route(cfg, x=d["x"], w_router=d["w_router"], logit_bias=d["logit_bias"])
    offsets, perm, dest, _ = moe.permute(cfg, ids, want_x_perm=False)
    y, _ = moe.mx_grouped_ffn(cfg, d["x"], dest, offsets, **q)
    a = M.values64(*moe.mx_quantize(d["x"], tiled=False))[perm.long()]
    off = offsets.tolist()
    ref = torch.zeros(y.shape, dtype=torch.float64, device=DEV)
    for e in range(cfg.E):
        s = slice(off[e], off[e + 1])
        if s.start == s.stop:
            continue
        w13 = M.values64(q["w13"][0][e], M.untile(q["w13"][1][e]))
        w2 = M.values64(q["w2"][0][e], M.untile(q["w2"][1][e]))
        g, u = (a[s] @ w13.T).chunk(2, 1)
        h = (g * torch.sigmoid(g) * u).to(torch.bfloat16)
        code, sc = M.quantize64(h)
        ref[s] = M.values64(M.pack(code), sc) @ w2.T
    err = (y.double() - ref).abs()
    assert (err.amax(1) / ref.abs().amax(1)).max() < 2.0 ** -5
    assert (err.mean() / ref.abs().mean()) < 2.0 ** -8


def test_tokens_keep_their_bits_in_any_batch():
    cfg, d, q, _ = layer("qwen3_30b_a3b", 400)
    kw = dict(logit_bias=d["logit_bias"])
    full = moe.mx_forward(cfg, d["x"], d["w_router"], **q, **kw)
    for sel in (slice(0, 1), slice(37, 165), torch.randperm(400, device=DEV)):
        x = d["x"][sel].contiguous()
        part = moe.mx_forward(cfg.with_T(x.shape[0]), x, d["w_router"], **q, **kw)
        assert eq(part, full[sel])


def test_tokens_keep_their_bits_across_the_row_tiles():
    """1100 tokens have 68 rows an expert on average, 500 and 1 have fewer than 64."""
    cfg, d, q, _ = layer("qwen3_30b_a3b", 1100)
    kw = dict(logit_bias=d["logit_bias"])
    full = moe.mx_forward(cfg, d["x"], d["w_router"], **q, **kw)
    for sel in (slice(3, 4), slice(600, 1100)):
        x = d["x"][sel].contiguous()
        part = moe.mx_forward(cfg.with_T(x.shape[0]), x, d["w_router"], **q, **kw)
        assert eq(part, full[sel])


def test_layer_replayed_from_a_graph_and_on_two_streams():
    cfg, d, q, _ = layer("qwen3_30b_a3b", 96)
    kw = dict(logit_bias=d["logit_bias"], check=False)
    x = d["x"].clone()
    st = moe.new_status(DEV)
    ws = torch.empty(moe.workspace_bytes(cfg, N.MOE_STAGE_MX_FORWARD), dtype=torch.uint8,
                     device=DEV)
    out = torch.empty_like(x)

    def call():
        moe.mx_forward(cfg, x, d["w_router"], **q, out=out, ws=ws, status=st, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    x2 = synthetic.normal_bf16(96, cfg.H, 1.0, 77, "x", device=DEV)
    want = [moe.mx_forward(cfg, v, d["w_router"], **q, **kw) for v in (d["x"], x2)]
    for v, ref in zip((d["x"], x2), want):
        x.copy_(v)
        graph.replay()
        assert eq(out, ref)
    moe.check_status(st)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s, v in zip(streams, (d["x"], x2)):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs += [moe.mx_forward(cfg, v, d["w_router"], **q, **kw) for _ in range(5)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert eq(o, want[i // 5])


class MadeWhenAsked:
    """Weights of mx_weight() as a sequence that makes its members anew each time."""

    def __init__(self, pair):
        self.pair = [t.cpu() for t in pair]

    def __len__(self):
        return 2

    def __getitem__(self, i):
        return self.pair[i].to(DEV)


def test_weights_from_a_sequence_are_held_through_the_call():
    """Nothing but the call refers to the members: their memory is not taken by its outputs."""
    cfg = moe.Config(T=70, H=256, E=4, K=2, I=128)
    x, wr = rows_like((70, 256), 1), rows_like((4, 256), 2)
    w13, w2 = moe.mx_weight(rows_like((4, 256, 256), 3)), moe.mx_weight(rows_like((4, 256, 128), 4))
    want, b = moe.mx_forward(cfg, x, wr, w13, w2, keep=True)
    got, _ = moe.mx_forward(cfg, x, wr, MadeWhenAsked(w13), MadeWhenAsked(w2), keep=True)
    assert eq(got, want)
    offsets, _, dest, _ = moe.permute(cfg, b["topk_ids"], want_x_perm=False)
    y, _ = moe.mx_grouped_ffn(cfg, x, dest, offsets, w13, w2)
    y2, _ = moe.mx_grouped_ffn(cfg, x, dest, offsets, MadeWhenAsked(w13), MadeWhenAsked(w2))
    assert eq(y, y2)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("bad", [[0, 40, 30, 60], [0, 300, 10, 500], [0, 300, -5, 500],
                                 [200, 600, 100, 350], [0, 900, 0, 600], [900, 40, 20, 10],
                                 [0, 128, 100, 260], [0, 10, 5, 7]])
def test_falling_offsets_give_the_clamped_groups(bad, glu):
    """Every offset clamped to the rows and raised to the largest before it: the results of those
    offsets, bit for bit and again, rows outside them as they were, and one count or more."""
    n, K, R = 512, 256, 600
    x, w = rows_like((R, K), 11), moe.mx_weight(rows_like((3, n, K), 12) * 0.02)
    q = moe.mx_quantize(x)
    good, top = [], 0
    for o in bad:
        top = max(top, min(max(o, 0), R))
        good.append(top)

    def run(off):
        out, st = torch.full((R, n // (1 + glu)), 3.0, dtype=torch.bfloat16, device=DEV), \
            moe.new_status(DEV)
        moe.mx_grouped_gemm(*q, torch.tensor(off, dtype=torch.int32, device=DEV), *w, swiglu=glu,
                            out=out, status=st, check=False)
        return out, st.tolist()

    want, clean = run(good)
    assert not any(clean)
    for _ in range(3):
        got, st = run(bad)
        assert eq(got, want) and st[N.MOE_ST_BAD_ROWS] > 0
        assert not any(v for i, v in enumerate(st) if i != N.MOE_ST_BAD_ROWS)


def test_falling_offsets_among_many_groups():
    """More groups than a block has threads, offsets that fall at several places among them."""
    groups, R = 700, 2000
    x, w = rows_like((R, 128), 13), moe.mx_weight(rows_like((groups, 128, 128), 14))
    q = moe.mx_quantize(x)
    off = [3 * g - (400 if g % 97 == 50 else 0) for g in range(groups)] + [R]
    good, top = [], 0
    for o in off:
        top = max(top, min(max(o, 0), R))
        good.append(top)
    a, b = (moe.mx_grouped_gemm(*q, torch.tensor(o, dtype=torch.int32, device=DEV), *w,
                                out=torch.zeros(R, 128, dtype=torch.bfloat16, device=DEV),
                                check=False) for o in (off, good))
    assert eq(a, b)
