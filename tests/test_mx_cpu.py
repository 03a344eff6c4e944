"""CPU checks of the 4-bit experts: the reference format by hand-worked values, the scale tiles,
and the refusals of the C ABI and the binding."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import mx_ref as M
from deterministic_invariant_routing_b200 import _native as N
from deterministic_invariant_routing_b200 import build, moe


@pytest.fixture(scope="module")
def lib():
    build.build()
    return N.load()


def test_reference_format_by_hand():
    x = torch.zeros(1, 32)
    # amax 6.9: exponent 2, scale 2^0; ties 0.25 0.75 1.25 1.75 2.5 3.5 5 go to even codes
    x[0, :16] = torch.tensor([6.9, -6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, 0.2501,
                              5.01, 4.99, -3.6, 0.0, 1.0])
    code, scale = M.quantize64(x)
    assert scale.tolist() == [[127]]
    assert code[0, :16].tolist() == [7, 15, 6, 6, 4, 4, 2, 2, 0, 8, 1, 7, 6, 14, 0, 2]
    v = M.values64(M.pack(code), scale)[0, :16].tolist()
    assert v == [6, -6, 4, 4, 2, 2, 1, 1, 0, 0, 0.5, 6, 4, -4, 0, 1]
    # scales: amax 2^k has exponent k - 2; zero and tiny blocks clamp at 2^-127
    for k in (-130, -126, -125, -124, 0, 5, 127):
        y = torch.zeros(1, 32, dtype=torch.float64)
        y[0, 3] = 2.0 ** k
        code, scale = M.quantize64(y)
        assert scale.item() == max(k - 2, -127) + 127
        if k >= -125:
            assert M.values64(M.pack(code), scale)[0, 3] == 2.0 ** k
    assert M.quantize64(torch.zeros(1, 32))[1].item() == 0


def test_scale_tiles_round_trip_and_layout():
    s = torch.arange(2 * 256 * 8, dtype=torch.int64).remainder(251).to(torch.uint8)
    s = s.view(2, 256, 8)
    t = M.tile(s)
    assert t.shape == (2, 2, 2, 512)
    for (e, r, b) in ((0, 0, 0), (0, 1, 0), (0, 33, 5), (1, 128 + 97, 7), (1, 255, 3)):
        assert t[e, r // 128, b // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4] == s[e, r, b]
    assert torch.equal(M.untile(t), s)


FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)


def test_quantize_refusals(lib):
    def q(rows=4, K=64, dt=0, tiled=0, x=FAKE, c=FAKE, s=FAKE):
        return lib.moe_mx_quantize(rows, K, dt, tiled, x, c, s, None)

    for over in (dict(rows=-1), dict(K=0), dict(K=48), dict(K=1 << 21), dict(dt=3), dict(dt=-1),
                 dict(rows=1 << 40, K=64)):
        assert q(**over) == N.MOE_ERR_SHAPE, over
    for over in (dict(tiled=2), dict(x=None), dict(c=None), dict(s=None), dict(x=ODD), dict(c=ODD),
                 dict(s=ODD, tiled=1)):
        assert q(**over) == N.MOE_ERR_ARG, over
    assert q(rows=0, x=None) == N.MOE_OK
    assert lib.moe_mx_dequantize(4, 48, 0, 0, FAKE, FAKE, FAKE, None) == N.MOE_ERR_SHAPE
    assert lib.moe_mx_dequantize(4, 64, 5, 0, FAKE, FAKE, FAKE, None) == N.MOE_ERR_SHAPE
    assert lib.moe_mx_dequantize(4, 64, 0, 1, FAKE, None, FAKE, None) == N.MOE_ERR_ARG
    assert lib.moe_mx_dequantize(4, 64, 0, 0, ODD, FAKE, FAKE, None) == N.MOE_ERR_ARG


def test_product_refusals(lib):
    def g(rows=4, K=128, n=256, groups=2, glu=0, a=FAKE, sa=FAKE, o=FAKE, b=FAKE, sb=FAKE, out=FAKE):
        return lib.moe_mx_grouped_gemm(rows, K, n, groups, glu, a, sa, o, b, sb, out, None, None)

    for over in (dict(rows=-1), dict(rows=1 << 31), dict(K=64), dict(K=192), dict(K=32896),
                 dict(n=64), dict(n=200), dict(n=384, glu=1), dict(groups=0), dict(groups=1025),
                 dict(n=32896), dict(groups=1024, n=65536, glu=1, K=128) | dict(n=131072)):
        assert g(**over) == N.MOE_ERR_SHAPE, over
    for over in (dict(glu=2), dict(o=None), dict(a=None), dict(sa=None), dict(b=None),
                 dict(sb=None), dict(out=None), dict(a=ODD), dict(sa=ODD), dict(b=ODD),
                 dict(sb=ODD), dict(out=ODD)):
        assert g(**over) == N.MOE_ERR_ARG, over
    assert g(rows=0, a=None) == N.MOE_OK


def test_layer_refusals(lib):
    c = moe.Config(T=8, H=256, E=4, K=2, I=128).c()
    need = lib.moe_workspace_bytes(ctypes.byref(c), N.MOE_STAGE_MX_FFN)
    assert need >= 8 * 2 * (256 + 128) * 17 // 32

    def ffn(cfg=c, ws_bytes=need, **over):
        names = ["x", "dest_row", "offsets", "w13", "w13_sc", "w2", "w2_sc", "w13_s", "w13_s_sc",
                 "w2_s", "w2_s_sc", "y", "y_shared", "status", "ws"]
        p = {n: FAKE for n in names}
        p.update({n: None for n in names if "_s" in n and n not in ("w13_sc", "w2_sc")})
        p["status"] = FAKE
        p.update(over)
        return lib.moe_mx_grouped_ffn(ctypes.byref(cfg), *[p[n] for n in names], ws_bytes, None)

    for over in ({k: None} for k in ("x", "dest_row", "offsets", "w13", "w13_sc", "w2", "w2_sc", "y")):
        assert ffn(**over) == N.MOE_ERR_ARG, over
    for over in (dict(x=ODD), dict(w13=ODD), dict(w2_sc=ODD), dict(y=ODD)):
        assert ffn(**over) == N.MOE_ERR_ARG, over
    assert ffn(ws_bytes=need - 1) == N.MOE_ERR_WORKSPACE
    assert ffn(ws=None) == N.MOE_ERR_WORKSPACE
    assert ffn(cfg=moe.Config(T=8, H=100, E=4, K=2, I=128).c()) == N.MOE_ERR_SHAPE
    shared = moe.Config(T=8, H=256, E=4, K=2, I=128, I_shared=128).c()
    assert ffn(cfg=shared) == N.MOE_ERR_ARG
    need = lib.moe_workspace_bytes(ctypes.byref(c), N.MOE_STAGE_MX_FORWARD)
    args = [FAKE, FAKE, None, None, None, *[FAKE] * 4, *[None] * 4, FAKE, None, None, None, None,
            FAKE, FAKE]
    assert lib.moe_mx_forward(ctypes.byref(c), *args, need - 1, None) == N.MOE_ERR_WORKSPACE
    args[0] = None
    assert lib.moe_mx_forward(ctypes.byref(c), *args, need, None) == N.MOE_ERR_ARG


def test_binding_refusals(lib):
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    c, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 1, 512, dtype=torch.uint8)
    flat = torch.zeros(4, 4, dtype=torch.uint8)
    wc = torch.zeros(2, 256, 64, dtype=torch.uint8)
    ws = torch.zeros(2, 2, 1, 512, dtype=torch.uint8)
    off = torch.zeros(3, dtype=torch.int32)
    bad = [lambda: moe.mx_quantize(x[0]), lambda: moe.mx_quantize(x.double()),
           lambda: moe.mx_quantize(x.t()), lambda: moe.mx_quantize(x),  # not on a GPU
           lambda: moe.mx_weight(x), lambda: moe.mx_weight(x.int()),
           lambda: moe.mx_weight(torch.zeros(128, 192)),
           lambda: moe.mx_dequantize(c, s, torch.int8), lambda: moe.mx_dequantize(c, flat[:, :3]),
           lambda: moe.mx_dequantize(c[:, :8].contiguous(), s),
           lambda: moe.mx_grouped_gemm(c, s, off[:2], wc, ws),
           lambda: moe.mx_grouped_gemm(c, s, off, wc, ws.flatten(2)),
           lambda: moe.mx_grouped_gemm(c, s.int(), off, wc, ws),
           lambda: moe.mx_grouped_gemm(c, flat, off, wc, ws),  # row-major scales
           lambda: moe.mx_grouped_gemm(c, s, off, wc[:, :128].contiguous(), ws, swiglu=True),
           lambda: moe.mx_grouped_gemm(c, s, off.long(), wc, ws),
           lambda: moe.mx_grouped_ffn(moe.Config(T=4, H=128, E=2, K=1, I=128), x,
                                      off[:2].view(2, 1), off, (wc, ws), (wc, ws)),
           lambda: moe.mx_grouped_ffn(moe.Config(T=4, H=128, E=2, K=1, I=128), x,
                                      torch.zeros(4, 1, dtype=torch.int32), off, (wc, ws), wc)]
    for f in bad:
        with pytest.raises(moe.MoeError):
            f()


def layer_on_the_cpu():
    """A small layer's arguments in host memory, and the bytes of its workspaces."""
    cfg = moe.Config(T=4, H=128, E=2, K=1, I=128)
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    w13 = (torch.zeros(2, 256, 64, dtype=torch.uint8), torch.zeros(2, 2, 1, 512, dtype=torch.uint8))
    w2 = (torch.zeros(2, 128, 64, dtype=torch.uint8), torch.zeros(2, 1, 1, 512, dtype=torch.uint8))
    dest, off = torch.zeros(4, 1, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    wr = torch.zeros(2, 128, dtype=torch.bfloat16)
    b13, b2 = (torch.zeros(2, n, 128, dtype=torch.bfloat16) for n in (256, 128))
    return cfg, x, w13, w2, dest, off, wr, b13, b2


def test_workspaces_that_are_no_buffer_of_the_device_are_refused(lib):
    """On another device than the call's tensors, strided, or expanded from fewer bytes."""
    cfg, x, w13, w2, dest, off, wr, b13, b2 = layer_on_the_cpu()
    n = 1 << 22
    wrong = [torch.empty(n, dtype=torch.uint8, device="meta"),
             torch.empty(2 * n, dtype=torch.uint8)[::2],
             torch.empty(1, dtype=torch.uint8).expand(n)]
    given = {"logits": torch.zeros(4, 2), "topk_ids": dest, "topk_w": torch.zeros(4, 1),
             "dout": x}
    for ws in wrong:
        for f in (lambda: moe.mx_grouped_ffn(cfg, x, dest, off, w13, w2, ws=ws),
                  lambda: moe.mx_forward(cfg, x, wr, w13, w2, ws=ws),
                  lambda: moe.forward(cfg, x, wr, b13, b2, ws=ws),
                  lambda: moe.forward_train(cfg, x, wr, b13, b2, ws),
                  lambda: moe.backward(cfg, x, wr, b13, b2, *given.values(), ws=ws),
                  lambda: moe.forward_host(cfg, x, wr, b13, b2, out_host=x, ws=ws)):
            with pytest.raises(moe.MoeError, match="workspace"):
                f()
    for f in (lambda ws: moe.mx_grouped_ffn(cfg, x, dest, off, w13, w2, ws=ws),
              lambda ws: moe.forward(cfg, x, wr, b13, b2, ws=ws)):
        with pytest.raises(moe.MoeError, match="workspace of 16 bytes"):
            f(torch.empty(16, dtype=torch.uint8))


def test_status_words_that_are_no_buffer_of_the_device_are_refused(lib):
    """On another device, of another type, too few, strided or expanded."""
    cfg, x, w13, w2, dest, off, wr, b13, b2 = layer_on_the_cpu()
    n = N.MOE_STATUS_WORDS
    wrong = [torch.zeros(n, dtype=torch.int32, device="meta"), torch.zeros(n),
             torch.zeros(n, dtype=torch.int64), torch.zeros(n - 1, dtype=torch.int32),
             torch.zeros(2 * n, dtype=torch.int32)[::2],
             torch.zeros(1, dtype=torch.int32).expand(n)]
    lg, tw = torch.zeros(4, 2), torch.zeros(4, 1)
    for st in wrong:
        for f in (lambda: moe.mx_forward(cfg, x, wr, w13, w2, status=st),
                  lambda: moe.mx_grouped_ffn(cfg, x, dest, off, w13, w2, status=st),
                  lambda: moe.mx_grouped_gemm(x.view(torch.uint8)[:, :64].contiguous(),
                                              w13[1][0, :1].contiguous(), off, *w13, status=st),
                  lambda: moe.route(cfg, x, wr, status=st),
                  lambda: moe.permute(cfg, dest, x, status=st),
                  lambda: moe.grouped_ffn(cfg, x, x, dest.view(-1), off, b13, b2, status=st),
                  lambda: moe.forward(cfg, x, wr, b13, b2, status=st),
                  lambda: moe.forward_train(cfg, x, wr, b13, b2,
                                            torch.empty(1 << 22, dtype=torch.uint8), status=st),
                  lambda: moe.backward(cfg, x, wr, b13, b2, lg, dest, tw, x, status=st),
                  lambda: moe.forward_host(cfg, x, wr, b13, b2, out_host=x, status=st)):
            with pytest.raises(moe.MoeError, match="status"):
                f()


HELD = """
import gc, sys
import torch
from deterministic_invariant_routing_b200 import moe
cfg = moe.Config(T=4, H=128, E=2, K=1, I=128)

class Weights:  # a sequence that makes its members when asked
    def __init__(self, n, k): self.n, self.k = n, k
    def __len__(self): return 2
    def __getitem__(self, i):
        if i > 1: raise IndexError(i)
        if i == 0: return torch.zeros(2, self.n, self.k // 2, dtype=torch.uint8)
        return torch.zeros(2, self.n // 128, self.k // 128, 512, dtype=torch.uint8)

x = torch.zeros(4, 128, dtype=torch.bfloat16)
dest, off = torch.zeros(4, 1, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
for _ in range(50):
    try:
        moe.mx_grouped_ffn(cfg, x, dest, off, Weights(256, 128), Weights(128, 128))
    except moe.MoeError as e:
        assert "tensors on cpu" in str(e), e
    else:
        sys.exit("not refused")
print("held")
"""


def test_weights_from_a_sequence_are_held_through_the_call(lib):
    """Members that only the call refers to: their shapes are read, and in a call on the GPU
    their memory is used, after the sequence's list of them is gone."""
    r = subprocess.run([sys.executable, "-c", HELD], capture_output=True, text=True,
                       cwd=os.path.dirname(build.PKG), env=dict(os.environ, PYTHONMALLOC="debug"))
    assert r.returncode == 0 and "held" in r.stdout, (r.returncode, r.stderr[-2000:])
