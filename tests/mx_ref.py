"""References of the microscaled 4-bit format and its products, in double (torch, any device)."""
from __future__ import annotations

import torch

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def pow2(e):
    """2^e exactly, e an integer tensor in [-1022, 1023]."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def quantize64(x):
    """(codes [..., K] one per byte, scales [..., K/32]) of finite x, straight from the format's
    definition: the nearest of the grid's values, found by comparing every distance; equal
    distances take the even code."""
    v = x.double().unflatten(-1, (-1, 32))
    amax = v.abs().amax(-1)
    # floor(log2(amax)) from the exponent bits of the double (0 for amax = 0: clamped below)
    e = ((amax.view(torch.int64) >> 52) - 1023 - 2).clamp(min=-127)
    a = v.abs() / pow2(e)[..., None]
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    dist = (a[..., None].clamp(max=6.0) - grid).abs()
    odd = torch.arange(8, device=x.device) % 2
    best = dist.amin(-1, keepdim=True)
    code = torch.where(dist == best, odd * 8 + torch.arange(8, device=x.device), 99).argmin(-1)
    code = code + 8 * torch.signbit(v).long()
    return code.flatten(-2).to(torch.uint8), (e + 127).to(torch.uint8)


def pack(code):
    return code[..., 0::2] | code[..., 1::2] << 4


def unpack(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def values64(codes, scales):
    """Values of packed codes and row-major scales; scale 255 is NaN."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), dtype=torch.float64, device=codes.device)
    k = pow2(scales.long() - 127)
    k = torch.where(scales == 255, float("nan"), k)
    return (grid[unpack(codes).long()].unflatten(-1, (-1, 32)) * k[..., None]).flatten(-2)


def tile(scales):
    """Row-major scales [..., N, K/32] in tiles [..., N/128, K/128, 512]."""
    *lead, n, b = scales.shape
    t = scales.view(-1, n // 128, 4, 32, b // 4, 4).permute(0, 1, 4, 3, 2, 5)
    return t.reshape(*lead, n // 128, b // 4, 512)


def untile(tiled):
    *lead, n, b, _ = tiled.shape
    t = tiled.view(-1, n, b, 32, 4, 4).permute(0, 1, 4, 3, 2, 5)
    return t.reshape(*lead, n * 128, b * 4)


def rows_of(tiled, R, K):
    """Row-major scales [R, K/32] from the tiles of [R, K] (padding dropped)."""
    return untile(tiled)[:R, :K // 32]


def product64(a, w, offsets, swiglu):
    """(out, magnitude of the sums) over groups of rows; NaN-free inputs. With swiglu both are
    of silu(gate) * up, its magnitude the first-order propagation of the sums'."""
    N = w.shape[1]
    v = a.new_zeros(a.shape[0], N)
    m = a.new_zeros(a.shape[0], N)
    for g in range(w.shape[0]):
        s = slice(offsets[g], offsets[g + 1])
        v[s] = a[s] @ w[g].T
        m[s] = a[s].abs() @ w[g].abs().T
    if not swiglu:
        return v, m
    g, u = v.chunk(2, 1)
    gm, um = m.chunk(2, 1)
    silu = g * torch.sigmoid(g)
    return silu * u, 1.1 * u.abs() * gm + silu.abs() * um
