"""Blocks of the layer end to end on the GPU: served with bf16 and 4-bit experts, and trained.
A block gives the bits of the calls it is made of, and its gradients, taken through two blocks
and the norm before them, agree with the 64-bit ones of the same computation."""
import numpy as np
import pytest
import torch

import block_ref as R
from deterministic_invariant_routing_b200 import moe, synthetic
from helpers import DEV
from oracle import backward64 as B

pytestmark = pytest.mark.gpu


def eq(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def stack(T, p, name="tiny", **over):
    """Two blocks over different layers, the first norm's weight and a residual stream."""
    g = torch.Generator(device=DEV).manual_seed(T)
    s0, d0 = synthetic.make_layer(name, T=T, device=DEV, **over)
    cfg = moe.Config.of(s0)
    d1 = {k: None if v is None else (v.roll(1, 0) if k != "x" else v) for k, v in d0.items()}

    def vec(scale=0.2):
        return 1 + scale * torch.randn(cfg.H, generator=g, device=DEV)

    blocks = []
    for d in (d0, d1):
        w = {k: d[k] for k in ("w_router", "w13", "w2", "logit_bias", "sel_bias", "w13_s", "w2_s")
             if d.get(k) is not None}
        blocks.append(moe.MoEBlock(moe.MoELayer(cfg, w), w_post=vec(), gate=vec(0.5),
                                   w_next=vec(), residual_scale=0.9, branch_scale=0.8, p=p))
    x = torch.randn(T, cfg.H, generator=g, device=DEV).bfloat16()
    return cfg, blocks, vec(), x


@pytest.mark.parametrize("name,T", [("tiny", 1), ("tiny", 61), ("qwen3_30b_a3b", 17)])
@pytest.mark.parametrize("mx", [False, True])
def test_served_blocks_equal_their_calls(name, T, mx):
    cfg, blocks, w0, x = stack(T, 0.0, name)
    if mx:
        for b in blocks:
            b.layer = b.layer.quantized()
            assert b.layer.mx and b.layer.quantized() is b.layer
    r, n = moe.residual_norm(x, w_next=w0)
    r2, n2 = r, n
    for b in blocks:
        r, n = b(r, n)
        w = b.layer.w
        f = moe.mx_forward if mx else moe.forward
        y = f(cfg, n2, w["w_router"], w["w13"], w["w2"], logit_bias=w.get("logit_bias"))
        r2, _ = moe.residual_norm(r2, y, **{**b.kw, "w_next": None})
        _, n2 = moe.residual_norm(r2, w_next=b.kw["w_next"])
        assert eq(r, r2) and eq(n, n2)


def test_layers_with_4_bit_experts_refuse_what_they_lack():
    cfg, blocks, w0, x = stack(8, 0.0)
    q = moe.MoEBlock(blocks[0].layer.quantized())
    n = x
    with pytest.raises(moe.MoeError, match="bf16 experts"):
        q.forward_train(x, n, moe.backward_workspace(cfg, DEV))
    with pytest.raises(moe.MoeError, match="bf16 experts"):
        q.layer.forward_host(x.cpu())
    with pytest.raises(moe.MoeError, match="stage events"):
        q.layer(n, stage_events=[None] * 8)


def test_trained_blocks_against_64_bits():
    """Loss = sum(c_r r + c_n n) after two blocks. The 64-bit gradients follow the GPU's stored
    tensors (its r, y and routes), so each operator is compared on the inputs it had: bf16
    gradients by row within 2^-5 of the row's largest (the layer's own bar is 2e-2; a seam adds
    two bf16 roundings, 2^-7, of it), parameter gradients within 2^-6 of their norm."""
    T, p = 61, 0.25
    cfg, blocks, w0, x = stack(T, p)
    rng = [moe.rng_state(7, i, device=DEV) for i in range(2)]
    r, n = moe.residual_norm(x, w_next=w0)
    saved = []
    for b, g in zip(blocks, rng):
        r, n, s = b.forward_train(r, n, moe.backward_workspace(cfg, DEV), rng=g)
        saved.append(s)
    gen = torch.Generator(device=DEV).manual_seed(1)
    dr = torch.randn(T, cfg.H, generator=gen, device=DEV).bfloat16()
    dn = torch.randn(T, cfg.H, generator=gen, device=DEV).bfloat16()
    got = []
    d = dict(dr=dr, dn=dn)
    for b, s in zip(reversed(blocks), reversed(saved)):
        g = b.backward(s, **d)
        got.insert(0, g)
        d = dict(dr=g["dx"], dn=g["dn"])
    first = moe.residual_norm_backward(x, w_next=w0, **d)

    def f64(t):
        return None if t is None else t.double()

    def rows(a, ref, what):
        e = (a.double() - ref).abs().amax(1) / ref.abs().amax(1)
        assert e.max() < 2.0 ** -5, (what, e.max().item())

    dr64, dn64 = dr.double(), dn.double()
    for i in (1, 0):
        b, s, g = blocks[i], saved[i], got[i]
        mask = R.scaled_mask(torch.arange(T, device=DEV), cfg.H, p, 7, i)
        ref = R.backward64(f64(s["r"]), f64(s["y"]), dr64, dn64, f64(b.kw["w_post"]),
                           f64(b.kw["gate"]), f64(b.kw["w_next"]), mask, b.kw["eps"], 0.9, 0.8)
        rows(g["dx"], ref["dx"][0], f"dx {i}")
        for k in ("dw_post", "dgate", "dw_next"):
            e = (g[k].double() - ref[k][0]).norm() / ref[k][0].norm()
            assert e < 2.0 ** -6, (k, i, e.item())
        w, rt = b.layer.w, s["routes"]
        lay = B.layer_backward64(*[v.double().cpu().numpy() for v in
                                   (ref["dy"][0], s["n"], w["w_router"], w["w13"], w["w2"])],
                                 rt["topk_ids"].cpu().numpy(), cfg.score_fn, cfg.renorm,
                                 cfg.route_scale)
        ref_dn = torch.from_numpy(np.asarray(lay["dx"])).to(DEV)
        rows(g["dn"], ref_dn, f"dn {i}")
        dr64, dn64 = ref["dx"][0], ref_dn
    ref = R.backward64(x.double(), None, dr64, dn64, None, None, w0.double(), None, 1e-6, 1.0, 1.0)
    rows(first["dx"], ref["dx"][0], "first dx")
    e = (first["dw_next"].double() - ref["dw_next"][0]).norm() / ref["dw_next"][0].norm()
    assert e < 2.0 ** -6


def test_training_step_is_bitwise_repeatable():
    cfg, blocks, w0, x = stack(33, 0.1)
    rng = moe.rng_state(3, device=DEV)
    out = []
    for _ in range(2):
        r, n = moe.residual_norm(x, w_next=w0)
        r, n, s = blocks[0].forward_train(r, n, moe.backward_workspace(cfg, DEV), rng=rng)
        g = blocks[0].backward(s, dr=r, dn=n)
        out.append([r, n, *g.pop("layer").values(), *g.values()])
    for a, b in zip(*out):
        assert a is None or eq(a, b)
