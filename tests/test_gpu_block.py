"""The operators around the layer on the GPU: residual_norm and its backward, dropout.

Reference: block_ref, in double, from the same inputs. Tolerances, derived: an output of type t
is rounded once, off by at most eps(t) / 2 of its value; before that every value is an fp32
expression. A sum over a row has a depth of at most 16 (a thread's elements) + 5 (shuffle) + 32
(warps) roundings, the rest of the chain fewer than 11: 64 roundings of 2^-24 relative to the
sum of the terms' magnitudes bound both (the norms divide by a root of such a sum, which halves
it). A parameter gradient adds rows of a group (at most ceil(T / groups)), groups / 16 partials
and 16 slices to that; T <= 4200 here keeps the depth below 64 + 80 + 74 + 16 < 256.
n is compared with the norm of the r that the GPU returned, its definition."""
import numpy as np
import pytest
import torch

import block_ref as R
from deterministic_invariant_routing_b200 import moe
from helpers import DEV

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def half(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps  # half the subnormal spacing, x2


def make(T, H, dt, gate="none", post=True, nxt=True, seed=0, params=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed + 31 * T + H)

    def rand(*s, d=dt, scale=1.0):
        return (torch.randn(*s, generator=g, device=DEV) * scale).to(d)

    v = {"x": rand(T, H), "y": rand(T, H, scale=0.5), "r": rand(T, H), "dr": rand(T, H),
         "dn": rand(T, H) if nxt else None, "w_post": (1 + rand(H, d=torch.float32, scale=0.2))
         .to(params) if post else None,
         "w_next": (1 + rand(H, d=torch.float32, scale=0.2)).to(params) if nxt else None,
         "gate": None}
    if gate != "none":
        v["gate"] = rand(*{"channel": (H,), "token": (T, 1), "full": (T, H)}[gate],
                         d=dt if gate == "full" else params)
    return v


def d64(t):
    return None if t is None else t.double()


def mask_of(T, H, p, seed, offset, first_row=0, row_ids=None):
    if p == 0:
        return None
    rows = torch.arange(first_row, first_row + T, device=DEV) if row_ids is None \
        else row_ids.long() & 0xFFFFFFFF
    return R.scaled_mask(rows, H, p, seed, offset)


def check(got, ref, mag, dt, name, depth=64):
    tol = half(dt) * ref.abs() + depth * U * mag * (1 + half(dt)) + tiny(dt)
    err = (got.double() - ref).abs()
    worst = (err / tol.clamp(min=1e-300)).max().item() if err.numel() else 0.0
    assert torch.isfinite(got).all() and worst <= 1.0, f"{name}: {worst:.3f} of the tolerance"


SHAPES = [(1, 8), (2, 64), (37, 72), (5, 256), (131, 264), (64, 512), (33, 520), (1021, 1000),
          (300, 2048), (7, 4096), (129, 4104), (3, 8192), (4, 8200), (3, 16384)]
MODES = [("none", True, True, 0.0), ("channel", True, True, 0.1), ("token", True, True, 0.5),
         ("full", True, True, 0.25), ("full", False, True, 0.0), ("token", False, False, 0.3),
         ("channel", True, False, 0.0), ("none", False, False, 0.0)]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("T,H", SHAPES)
def test_residual_norm_and_backward(dt, T, H):
    dtype = TYPES[dt]
    for m, (gate, post, nxt, p) in enumerate(MODES):
        params = dtype if m % 2 else torch.float32
        v = make(T, H, dtype, gate, post, nxt, seed=m, params=params)
        rng = moe.rng_state(2 ** 40 + m, 2 ** 33 + 5, device=DEV)
        mask = mask_of(T, H, p, 2 ** 40 + m, 2 ** 33 + 5)
        kw = dict(w_post=v["w_post"], gate=v["gate"], w_next=v["w_next"], eps=EPS,
                  residual_scale=0.75, branch_scale=-1.25, p=p, rng=rng)
        r, n = moe.residual_norm(v["x"], v["y"], **kw)
        ref, mag = R.forward64(d64(v["x"]), d64(v["y"]), d64(v["w_post"]), d64(v["gate"]), mask,
                               EPS, 0.75, -1.25)
        check(r, ref, mag, dtype, f"r {gate} {post} {p}")
        if nxt:
            ref = R.norm64(r.double(), d64(v["w_next"]), EPS)
            check(n, ref, ref.abs(), dtype, f"n {gate}")
        else:
            assert n is None
        got = moe.residual_norm_backward(v["r"], v["y"], dr=v["dr"], dn=v["dn"], **kw)
        refs = R.backward64(d64(v["r"]), d64(v["y"]), d64(v["dr"]), d64(v["dn"]), d64(v["w_post"]),
                            d64(v["gate"]), d64(v["w_next"]), mask, EPS, 0.75, -1.25)
        assert set(got) == set(refs)
        for name, (g, gm) in refs.items():
            out = got[name]
            want = dtype if name in ("dx", "dy") or (name == "dgate" and gate == "full") \
                else torch.float32
            assert out.dtype == want and out.shape == g.shape
            check(out, g, gm, want, f"{name} {gate} {post} {p}", depth=256)


@pytest.mark.parametrize("gate,p", [("channel", 0.2), ("channel", 0.0), ("full", 0.2),
                                    ("token", 0.2)])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("T,H", [(700, 128), (650, 200), (401, 400), (500, 1000), (333, 2048),
                                 (310, 4000), (350, 6008), (12, 8192), (9, 8408)])
def test_backward_of_the_usual_call(dt, T, H, gate, p):
    """Both norms, fp32 parameters and dr, in rows that fill their threads and that do not."""
    v = make(T, H, TYPES[dt], gate, seed=3)
    rng = moe.rng_state(4, 4, device=DEV)
    kw = dict(w_post=v["w_post"], gate=v["gate"], w_next=v["w_next"], eps=EPS,
              residual_scale=0.75, branch_scale=1.5, p=p, rng=rng)
    if gate == "channel":
        kw["gate"] = v["gate"] = v["gate"].float()
    got = moe.residual_norm_backward(v["r"], v["y"], dr=v["dr"], dn=v["dn"], **kw)
    refs = R.backward64(d64(v["r"]), d64(v["y"]), d64(v["dr"]), d64(v["dn"]), d64(v["w_post"]),
                        d64(v["gate"]), d64(v["w_next"]), mask_of(T, H, p, 4, 4), EPS, 0.75, 1.5)
    assert set(got) == set(refs)
    for name, (g, gm) in refs.items():
        check(got[name], g, gm, got[name].dtype, name, depth=256)


@pytest.mark.parametrize("dt", list(TYPES))
def test_norm_alone(dt):
    """Without y: the norm before the first block, and its gradients with and without dr."""
    for T, H in ((1, 2048), (77, 136), (4200, 512)):
        v = make(T, H, TYPES[dt])
        r, n = moe.residual_norm(v["x"], w_next=v["w_next"])
        assert r is v["x"]
        ref = R.norm64(d64(v["x"]), d64(v["w_next"]), EPS)
        check(n, ref, ref.abs(), TYPES[dt], "n")
        for dr in (None, v["dr"]):
            got = moe.residual_norm_backward(v["x"], dr=dr, dn=v["dn"], w_next=v["w_next"])
            refs = R.backward64(d64(v["x"]), None, d64(dr), d64(v["dn"]), None, None,
                                d64(v["w_next"]), None, EPS, 1.0, 1.0)
            assert set(got) == {"dx", "dw_next"}
            for name, (g, gm) in refs.items():
                check(got[name], g, gm, TYPES[dt] if name == "dx" else torch.float32, name, 256)


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy().tobytes()


@pytest.mark.parametrize("H", [64, 2048, 8192])
def test_rows_do_not_depend_on_the_batch(H):
    """A row's r, n, dx, dy and token gate gradient have the same bits alone, in a chunk, or
    permuted, when its row number travels with it; repeated calls give the same bits for all."""
    T, p = 203, 0.3
    v = make(T, H, torch.bfloat16, "token")
    rng = moe.rng_state(9, 1, device=DEV)
    base = dict(w_post=v["w_post"], w_next=v["w_next"], p=p, rng=rng)

    def both(sel, **rows):
        kw = dict(base, gate=v["gate"][sel].contiguous(), **rows)
        r, n = moe.residual_norm(v["x"][sel], v["y"][sel], **kw)
        return r, n, moe.residual_norm_backward(v["r"][sel], v["y"][sel], dr=v["dr"][sel],
                                                dn=v["dn"][sel], **kw)

    r, n, g = both(slice(None))
    r2, n2, g2 = both(slice(None))
    assert raw(r) == raw(r2) and raw(n) == raw(n2) and all(raw(g[k]) == raw(g2[k]) for k in g)
    perm = torch.randperm(T, device=DEV)
    for sel, rows in ((slice(70, 71), dict(first_row=70)), (slice(31, 160), dict(first_row=31)),
                      (perm, dict(row_ids=perm.int()))):
        rs, ns, gs = both(sel, **rows)
        assert raw(rs) == raw(r[sel]) and raw(ns) == raw(n[sel])
        for k in ("dx", "dy", "dgate"):
            assert raw(gs[k]) == raw(g[k][sel]), k


MANY = [(520, *MODES[1]), (1000, *MODES[3]), (2048, *MODES[1]), (2048, "channel", True, True, 0.0),
        (2048, "none", True, True, 0.3), (4000, *MODES[2]), (4096, *MODES[4]), (4104, *MODES[1]),
        (5120, *MODES[3]), (1032, *MODES[5]), (2048, *MODES[6]), (8192, *MODES[1])]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_rows(dt, case):
    """Calls whose rows outnumber the blocks that are resident at once (at most 512 threads an
    SM, two vectors of 8 a thread): every row is right and has the bits it has in a call of few
    rows, with non-finite rows among them, and in place."""
    H, gate, post, nxt, p = MANY[case]
    dtype, threads = TYPES[dt], -(-H // 512) * 32
    T = 2 * 148 * (512 // threads) + 3
    v = make(T, H, dtype, gate, post, nxt, seed=case, params=dtype if case % 3 == 2 else
             torch.float32)
    rng = moe.rng_state(5, case, device=DEV)
    kw = dict(w_post=v["w_post"], w_next=v["w_next"], residual_scale=0.5, p=p, rng=rng)
    r, n = moe.residual_norm(v["x"], v["y"], gate=v["gate"], **kw)
    mask = mask_of(T, H, p, 5, case)
    ref, mag = R.forward64(d64(v["x"]), d64(v["y"]), d64(v["w_post"]), d64(v["gate"]), mask,
                           EPS, 0.5, 1.0)
    check(r, ref, mag, dtype, "r")
    if nxt:
        ref = R.norm64(r.double(), d64(v["w_next"]), EPS)
        check(n, ref, ref.abs(), dtype, "n")
        check(moe.residual_norm(v["x"], w_next=v["w_next"])[1],
              R.norm64(d64(v["x"]), d64(v["w_next"]), EPS),
              R.norm64(d64(v["x"]), d64(v["w_next"]), EPS).abs(), dtype, "norm alone")
    v["y"][7, 100], v["y"][T - 2, 3], v["x"][9, H - 1] = float("nan"), float("inf"), float("inf")
    r, n = moe.residual_norm(v["x"], v["y"], gate=v["gate"], **kw)
    for a, b in ((0, 1), (5, 105), (T - 40, T)):
        g = v["gate"] if v["gate"] is None or gate == "channel" else v["gate"][a:b].contiguous()
        r1, n1 = moe.residual_norm(v["x"][a:b], v["y"][a:b], gate=g, first_row=a, **kw)
        assert raw(r1) == raw(r[a:b]) and (not nxt or raw(n1) == raw(n[a:b]))
        if nxt:
            whole = moe.residual_norm(v["x"], w_next=v["w_next"])[1]
            assert raw(whole[a:b]) == raw(moe.residual_norm(v["x"][a:b], w_next=v["w_next"])[1])
    x, y = v["x"].clone(), v["y"].clone()
    moe.residual_norm(x, y, gate=v["gate"], r=x, n=y if nxt else None, **kw)
    assert raw(x) == raw(r) and (not nxt or raw(y) == raw(n))


def test_fused_call_equals_the_calls_it_replaces():
    """r then the norm of r; the branch's dropout as its own call; outputs in place."""
    T, H, p = 111, 1024, 0.4
    v = make(T, H, torch.float32, "none", post=False)
    rng = moe.rng_state(77, device=DEV)
    r, n = moe.residual_norm(v["x"], v["y"], w_next=v["w_next"], p=p, rng=rng)
    _, n2 = moe.residual_norm(r, w_next=v["w_next"])
    assert raw(n) == raw(n2)
    r3, none = moe.residual_norm(v["x"], moe.dropout(v["y"], p, rng))
    assert none is None and raw(r3) == raw(r)
    x, y = v["x"].clone(), v["y"].clone()
    moe.residual_norm(x, y, w_next=v["w_next"], p=p, rng=rng, r=x, n=y)
    assert raw(x) == raw(r) and raw(y) == raw(n)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("T,H,p", [(1, 8, 0.5), (333, 128, 0.5), (1000, 136, 0.1), (3, 16384, 0.9),
                                   (17, 24, 0.0), (17, 24, 2.0 ** -18), (9, 40, 1.0),
                                   (2049, 2048, 0.015)])
def test_dropout_values_and_mask(dt, T, H, p):
    """Every value: the fp32 product with the exact scale, rounded to the type, or +0."""
    x = torch.randn(T, H, device=DEV, generator=torch.Generator(device=DEV).manual_seed(T)) \
        .to(TYPES[dt])
    out = moe.dropout(x, p, moe.rng_state(2 ** 63 + 17, 3, device=DEV))
    f = R.scaled_mask(torch.arange(T, device=DEV), H, p, 2 ** 63 + 17, 3).float()
    ref = torch.where(f != 0, x.float() * f, 0.0).to(TYPES[dt])
    assert raw(out) == raw(ref)


def test_dropout_rows_and_gradient():
    """Rows by number: a chunk, a permutation, row numbers up to 2^32 - 1; the gradient is the
    same call; in place."""
    T, H, p = 50, 256, 0.35
    x = torch.randn(T, H, device=DEV)
    rng = moe.rng_state(4, 4, device=DEV)
    full = moe.dropout(x, p, rng)
    assert raw(moe.dropout(x[20:33], p, rng, first_row=20)) == raw(full[20:33])
    perm = torch.randperm(T, device=DEV)
    assert raw(moe.dropout(x[perm], p, rng, row_ids=perm.int())) == raw(full[perm])
    top = moe.dropout(x, p, rng, first_row=2 ** 32 - T)
    ids = torch.arange(-T, 0, dtype=torch.int32, device=DEV)
    assert raw(top) == raw(moe.dropout(x, p, rng, row_ids=ids))
    f = R.scaled_mask(torch.arange(2 ** 32 - T, 2 ** 32, device=DEV), H, p, 4, 4).float()
    assert raw(top) == raw(torch.where(f != 0, x * f, 0.0))
    d = torch.randn(T, H, device=DEV)
    f = R.scaled_mask(torch.arange(T, device=DEV), H, p, 4, 4).float()
    assert raw(moe.dropout(d, p, rng)) == raw(torch.where(f != 0, d * f, 0.0))
    y = x.clone()
    assert moe.dropout(y, p, rng, out=y) is y and raw(y) == raw(full)


def test_non_finite_values_stay_in_their_rows():
    """Dropped infinities and NaNs give 0; a NaN in a row leaves every other row's bits alone."""
    T, H, p = 40, 512, 0.5
    keep = R.keep_mask(torch.arange(T, device=DEV), H, p, 1, 0)
    x = torch.where(keep, 1.0, float("inf"))
    x[3] = torch.where(keep[3], 1.0, float("nan"))
    out = moe.dropout(x, p, moe.rng_state(1, device=DEV))
    assert torch.equal(out, keep.float() * 2)
    v = make(T, H, torch.bfloat16, "channel")
    kw = dict(w_post=v["w_post"], gate=v["gate"], w_next=v["w_next"])
    r0, n0 = moe.residual_norm(v["x"], v["y"], **kw)
    g0 = moe.residual_norm_backward(v["r"], v["y"], dr=v["dr"], dn=v["dn"], **kw)
    v["y"][7, 100] = float("nan")
    r1, n1 = moe.residual_norm(v["x"], v["y"], **kw)
    g1 = moe.residual_norm_backward(v["r"], v["y"], dr=v["dr"], dn=v["dn"], **kw)
    rest = torch.arange(T, device=DEV) != 7
    assert n1[7].isnan().all() and r1[7].isnan().all() and g1["dy"][7].isnan().all()
    for a, b in ((r0, r1), (n0, n1), (g0["dx"], g1["dx"]), (g0["dy"], g1["dy"])):
        assert raw(a[rest]) == raw(b[rest])
    z = torch.zeros(2, H, device=DEV)
    r, n = moe.residual_norm(z, z, w_post=torch.ones(H, device=DEV),
                             w_next=torch.ones(H, device=DEV))
    assert not r.any() and not n.any()


def test_no_rows():
    for H in (8, 2048):
        x = torch.zeros(0, H, device=DEV)
        w = torch.ones(H, device=DEV)
        r, n = moe.residual_norm(x, x, w_post=w, w_next=w, gate=w)
        assert r.shape == n.shape == (0, H)
        g = moe.residual_norm_backward(x, x, dr=x, dn=x, w_post=w, w_next=w, gate=w)
        assert not g["dw_post"].any() and not g["dw_next"].any() and not g["dgate"].any()
        assert moe.dropout(x, 0.5, moe.rng_state(1, device=DEV)).shape == (0, H)


def test_captured_step_draws_new_masks():
    """Forward and backward in one CUDA graph on a side stream; the owner of the generator
    state changes it between replays, and each replay equals the eager calls."""
    T, H, p = 65, 768, 0.2
    v = make(T, H, torch.bfloat16, "channel")
    rng = moe.rng_state(5, 0, device=DEV)
    kw = dict(w_post=v["w_post"], gate=v["gate"], w_next=v["w_next"], p=p, rng=rng)

    def step():
        r, n = moe.residual_norm(v["x"], v["y"], **kw)
        return r, n, moe.residual_norm_backward(r, v["y"], dr=v["dr"], dn=v["dn"], **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, n, g = step()
    seen = set()
    for offset in (0, 1, 2):
        rng.copy_(moe.rng_state(5, offset, device=DEV))
        graph.replay()
        got = [raw(t) for t in (r, n, *g.values())]
        r2, n2, g2 = step()
        assert got == [raw(t) for t in (r2, n2, *g2.values())]
        seen.add(got[0])
    assert len(seen) == 3


def test_more_than_two_to_the_31_elements():
    """Indices past 31 bits: the last rows equal a call on those rows alone."""
    T, H, p = 132000, 16384, 0.5
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    x[-9:] = torch.randn(9, H, device=DEV)
    tail = x[-9:].clone()
    rng = moe.rng_state(3, device=DEV)
    w = torch.rand(H, device=DEV)
    small = moe.dropout(tail, p, rng, first_row=T - 9)
    rs, ns = moe.residual_norm(tail, tail, w_post=w, w_next=w, p=p, rng=rng, first_row=T - 9)
    moe.dropout(x, p, rng, out=x)
    assert raw(x[-9:]) == raw(small)
    x[-9:] = tail
    y = x.clone()
    moe.residual_norm(x, y, w_post=w, w_next=w, p=p, rng=rng, r=x, n=y)
    assert raw(x[-9:]) == raw(rs) and raw(y[-9:]) == raw(ns)


@pytest.mark.parametrize("dt,H,gate", [("bf16", 520, "token"), ("bf16", 2048, "channel"),
                                       ("f32", 1000, "token"), ("f16", 4104, "full"),
                                       ("f32", 4096, "channel"), ("bf16", 8200, "none")])
def test_backward_repeats_its_bits(dt, H, gate):
    """Rows of several warps, many to a block, both reductions of each: call after call, beside
    other work on the GPU, every output has the same bits."""
    T = 1500
    v = make(T, H, TYPES[dt], gate, seed=8)
    rng = moe.rng_state(6, 6, device=DEV)
    kw = dict(w_post=v["w_post"], gate=v["gate"], w_next=v["w_next"], eps=EPS, p=0.1, rng=rng)
    first = moe.residual_norm_backward(v["r"], v["y"], dr=v["dr"], dn=v["dn"], **kw)
    other, side = torch.zeros(1 << 24, device=DEV), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for i in range(60):
        if i % 2:
            with torch.cuda.stream(side):
                other.add_(1.0)
        g = moe.residual_norm_backward(v["r"], v["y"], dr=v["dr"], dn=v["dn"], **kw)
        for k, t in g.items():
            differ += (t.view(torch.uint8) != first[k].view(torch.uint8)).sum()
    torch.cuda.current_stream().wait_stream(side)
    assert differ.item() == 0


# Roundings of a row's gradients, relative to the sum of their terms' magnitudes. A row's sum takes
# at most 8 fused adds a thread, 1 for the pair, 5 + 5 shuffles (19) and 2 for the mean; an inverse
# root half of its argument's 22 and 4 of its own (2 ulp): 15. The mean of w dn r: 23 with its two
# products; times three inverse roots and their products 71, times r and residual_scale 73: dx.
# The branch's gradient has three products more and the weight (77); its mean with y u takes 17 of
# y u and 21 of the sum (115), two inverse roots and products 147, times y 148 and one sum: dy.
# A token's gate: 77, 18 of z, 19 of the sum.
DEPTH = {"dx": 80, "dy": 160, "dgate": 120}


def check_rows(got, refs, skip=()):
    for name, (g, gm) in refs.items():
        if name in got and name not in skip and got[name].shape[0] == refs["dx"][0].shape[0]:
            check(got[name], g, gm, got[name].dtype, name, DEPTH[name])


@pytest.mark.parametrize("scale", [1e13, 1e15, 1e16])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", [128, 512, 1000, 2048, 4104, 8200])
def test_gradients_of_large_rows(dt, H, scale):
    """Rows whose inverse root is far from 1 (its cube is not an fp32 number any more), with a
    gradient along the row, so that the norm's projection is as large as the other term."""
    v = make(7, H, TYPES[dt], "token")
    x, y = d64(v["r"]), d64(v["y"])
    big, wide = (x * scale).to(TYPES[dt]), (y * scale).to(TYPES[dt])
    dn = (x + 0.1 * d64(v["dn"])).to(TYPES[dt])
    small = (d64(v["dr"]) / scale).to(TYPES[dt])
    for dr in (None, small):
        kw = dict(w_post=v["w_post"], gate=v["gate"].float(), w_next=v["w_next"], eps=EPS)
        got = moe.residual_norm_backward(big, wide, dr=dr, dn=dn, **kw)
        refs = R.backward64(d64(big), d64(wide), d64(dr) if dr is not None else None, d64(dn),
                            d64(v["w_post"]), d64(kw["gate"]), d64(v["w_next"]), None, EPS, 1.0,
                            1.0)
        check_rows({k: t for k, t in got.items() if k == "dx"}, refs)
        alone = moe.residual_norm_backward(big, dr=dr, dn=dn, w_next=v["w_next"])
        check_rows(alone, refs)
        got = moe.residual_norm_backward(v["r"], wide, dr=v["dr"], dn=dn, **kw)
        refs = R.backward64(d64(v["r"]), d64(wide), d64(v["dr"]), d64(dn), d64(v["w_post"]),
                            d64(kw["gate"]), d64(v["w_next"]), None, EPS, 1.0, 1.0)
        check_rows(got, refs)


@pytest.mark.parametrize("eps", [1e-30, 1e-40])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("H", [256, 520, 2048, 8200])
def test_gradients_of_zero_rows_with_a_small_eps(dt, H, eps):
    """A row of zeros has the inverse root eps^-1/2, 1e15 and more: its gradient is dn w times
    that, with no projection, never a NaN. (fp16 holds no such gradient: dn is 0 there.)"""
    T = 5
    v = make(T, H, TYPES[dt], "none")
    v["r"][2], v["y"][2] = 0, 0
    if dt == "f16":
        v["dn"][2], v["dr"][2] = 0, 0
    # only dx of the row is looked at where its gradient reaches dy through another 1 / sqrt(eps)
    got = moe.residual_norm_backward(v["r"], v["y"], dr=v["dr"], dn=v["dn"], w_post=v["w_post"],
                                     w_next=v["w_next"], eps=eps, branch_scale=0.0)
    eps = torch.tensor(eps, dtype=torch.float32).double().item()
    refs = R.backward64(d64(v["r"]), d64(v["y"]), d64(v["dr"]), d64(v["dn"]), d64(v["w_post"]),
                        None, d64(v["w_next"]), None, eps, 1.0, 0.0)
    check_rows(got, refs, skip=("dy",))
    assert not got["dy"].any()
    g = moe.residual_norm_backward(v["r"], v["y"], dr=v["dr"], w_post=v["w_post"], eps=eps,
                                   branch_scale=1e-12)
    refs = R.backward64(d64(v["r"]), d64(v["y"]), d64(v["dr"]), None, d64(v["w_post"]), None, None,
                        None, eps, 1.0, float(torch.tensor(1e-12)))
    check_rows(g, refs)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("T,H", SHAPES + [(700, 2048), (650, 200)])
def test_row_gradients_within_their_own_bounds(dt, T, H):
    """dx, dy and the gates' gradients of each row, under the roundings of a row alone (DEPTH),
    without what the sums over tokens add."""
    for m, (gate, post, nxt, p) in enumerate(MODES + [("token", True, True, 0.0)]):
        v = make(T, H, TYPES[dt], gate, post, nxt, seed=40 + m,
                 params=TYPES[dt] if m % 2 == 0 else torch.float32)
        rng = moe.rng_state(m, 2, device=DEV)
        got = moe.residual_norm_backward(v["r"], v["y"], dr=v["dr"], dn=v["dn"], eps=EPS,
                                         w_post=v["w_post"], gate=v["gate"], w_next=v["w_next"],
                                         residual_scale=0.75, branch_scale=-1.25, p=p, rng=rng)
        refs = R.backward64(d64(v["r"]), d64(v["y"]), d64(v["dr"]), d64(v["dn"]), d64(v["w_post"]),
                            d64(v["gate"]), d64(v["w_next"]), mask_of(T, H, p, m, 2), EPS, 0.75,
                            -1.25)
        check_rows(got, refs, skip=("dgate",) if gate == "channel" else ())
