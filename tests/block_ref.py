"""64-bit references of the operators around the layer (torch, any device): the counter-based
mask, the fused residual norm and its gradients."""
from __future__ import annotations

import math

import torch


def philox(counter, key):
    """Philox4x32-10 of int64 tensors (or ints) holding 32-bit words; products of 32 by 32 bits
    are formed from 16-bit halves, so nothing overflows."""
    c, k = list(counter), list(key)

    def mul(a, m):
        lo, hi = (a & 0xFFFF) * m, (a >> 16) * m
        low = lo + ((hi & 0xFFFF) << 16)
        return (hi >> 16) + (low >> 32), low & 0xFFFFFFFF

    for _ in range(10):
        h0, l0 = mul(c[0], 0xD2511F53)
        h1, l1 = mul(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k[0], l1, h0 ^ c[3] ^ k[1], l0]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p: float) -> int:
    return math.floor(p * 65536 + 0.5)


def keep_mask(rows: torch.Tensor, H: int, p: float, seed: int, offset: int) -> torch.Tensor:
    """[len(rows), H] bool: kept elements of these row numbers."""
    M = 0xFFFFFFFF
    row = rows.long()[:, None].expand(-1, H // 8)
    col = torch.arange(H // 8, device=rows.device)[None].expand_as(row)
    o = torch.zeros_like(row)
    w = philox([col, row, o + (offset & M), o + ((offset >> 32) & M)],
               [seed & M, (seed >> 32) & M])
    u = torch.stack([v for x in w for v in (x & 0xFFFF, x >> 16)], -1).reshape(len(rows), H)
    return u >= threshold(p)


def scaled_mask(rows, H, p, seed, offset):
    """The factor of each element, 0 or 1 / P(keep), in double."""
    t = threshold(p)
    k = keep_mask(rows, H, p, seed, offset)
    return k.double() * (65536.0 / (65536 - t) if t < 65536 else 0.0)


def _inv(v, eps):
    return (v.square().mean(-1, keepdim=True) + eps).rsqrt()


def forward64(x, y, w_post, gate, mask, eps, rs, bs):
    """(r, magnitude of its terms), double and unrounded."""
    z = y * _inv(y, eps) * w_post if w_post is not None else y
    if mask is not None:
        z = torch.where(mask != 0, z * mask, 0.0)
    if gate is not None:
        z = z * gate
    return rs * x + bs * z, (rs * x).abs() + (bs * z).abs()


def norm64(r, w, eps):
    return r * _inv(r, eps) * w


def _norm_grad(v, w, d, eps):
    """(dv, magnitude of its terms, dw terms) of rms(v) * w."""
    s = _inv(v, eps)
    m = (w * d * v).mean(-1, keepdim=True)
    mm = (w * d * v).abs().mean(-1, keepdim=True)
    return (s * w * d - v * s ** 3 * m, (s * w * d).abs() + (v * s ** 3).abs() * mm, d * v * s)


def backward64(r, y, dr, dn, w_post, gate, w_next, mask, eps, rs, bs):
    """{name: (gradient, magnitude of the terms it was summed from)}, double and unrounded."""
    out = {}
    d, dm = (dr, dr.abs()) if dr is not None else (torch.zeros_like(r), torch.zeros_like(r))
    if w_next is not None:
        dv, mag, dw = _norm_grad(r, w_next, dn, eps)
        d, dm = d + dv, dm + mag
        out["dw_next"] = (dw.sum(0), dw.abs().sum(0))
    out["dx"] = (rs * d, abs(rs) * dm)
    if y is None:
        return out
    b, bm = bs * d, abs(bs) * dm
    z = y * _inv(y, eps) * w_post if w_post is not None else y
    if mask is not None:
        z = torch.where(mask != 0, z * mask, 0.0)
    c, cm = b, bm
    if gate is not None:
        g, gm = b * z, bm * z.abs()
        if gate.dim() == 1:
            out["dgate"] = (g.sum(0), gm.sum(0))
        elif gate.shape[1] == 1:
            out["dgate"] = (g.sum(1, keepdim=True), gm.sum(1, keepdim=True))
        else:
            out["dgate"] = (g, gm)
        c, cm = c * gate, cm * gate.abs()
    if mask is not None:
        c, cm = torch.where(mask != 0, c * mask, 0.0), cm * mask
    if w_post is not None:
        s = _inv(y, eps)
        dw, dwm = c * y * s, cm * (y * s).abs()
        out["dw_post"] = (dw.sum(0), dwm.sum(0))
        dv, _, _ = _norm_grad(y, w_post, c, eps)
        _, mag, _ = _norm_grad(y, w_post.abs(), cm, eps)
        c, cm = dv, mag
    out["dy"] = (c, cm)
    return out
