"""CPU checks of the operators around the layer: the counter-based generator against its
published vectors, the reference gradients against central differences, and the refusals of
the C ABI and of the binding (no GPU and no CUDA call is reached)."""
import ctypes
import importlib.util
import subprocess
import sys

import pytest
import torch

import block_ref as R
from deterministic_invariant_routing_b200 import _native as N
from deterministic_invariant_routing_b200 import build, moe


@pytest.fixture(scope="module")
def lib():
    build.build()
    return N.load()


def test_philox_published_vectors():
    """The known-answer vectors of the generator's authors (10 rounds, 4 x 32)."""
    F = 0xFFFFFFFF
    assert R.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert R.philox([F] * 4, [F] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert R.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344],
                    [0xA4093822, 0x299F31D0]) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_mask_rate_and_independence():
    """The share kept is the threshold's probability within 5 standard deviations, over rows,
    columns, seeds and offsets; masks of different seeds, offsets or rows differ."""
    n, H = 512, 512
    rows = torch.arange(n)
    for p in (0.1, 0.5, 0.9):
        k = R.keep_mask(rows, H, p, 1234567, 8)
        q = 1 - R.threshold(p) / 65536
        sd = (q * (1 - q) / (n * H)) ** 0.5
        assert abs(k.double().mean() - q) < 5 * sd
        assert (k.double().mean(0) - q).abs().max() < 6 * (q * (1 - q) / n) ** 0.5
    a = R.keep_mask(rows, H, 0.5, 1, 0)
    for other in (R.keep_mask(rows, H, 0.5, 2, 0), R.keep_mask(rows, H, 0.5, 1, 1),
                  R.keep_mask(rows, H, 0.5, 1 << 32, 0), R.keep_mask(rows, H, 0.5, 1, 1 << 32),
                  R.keep_mask(rows + 1, H, 0.5, 1, 0)):
        assert 0.4 < (a == other).double().mean() < 0.6


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post,nxt,p", [(True, True, 0.3), (False, True, 0.0), (True, False, 0.5)])
def test_reference_gradients_against_differences(gate, post, nxt, p):
    """backward64 against central differences of forward64 / norm64, in double."""
    g = torch.Generator().manual_seed(3)
    T, H, eps, rs, bs = 3, 16, 1e-3, 0.7, 1.3

    def rand(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    v = {"x": rand(T, H), "y": rand(T, H)}
    if post:
        v["w_post"] = rand(H)
    if nxt:
        v["w_next"] = rand(H)
    if gate != "none":
        v["gate"] = rand(*{"channel": (H,), "token": (T, 1), "full": (T, H)}[gate])
    mask = R.scaled_mask(torch.arange(T), H, p, 5, 6) if p else None
    dr, dn = rand(T, H), rand(T, H) if nxt else None

    def loss(v):
        r, _ = R.forward64(v["x"], v["y"], v.get("w_post"), v.get("gate"), mask, eps, rs, bs)
        out = (r * dr).sum()
        return out + (R.norm64(r, v["w_next"], eps) * dn).sum() if nxt else out

    r, _ = R.forward64(v["x"], v["y"], v.get("w_post"), v.get("gate"), mask, eps, rs, bs)
    got = R.backward64(r, v["y"], dr, dn, v.get("w_post"), v.get("gate"), v.get("w_next"), mask,
                       eps, rs, bs)
    h = 1e-5
    for name, t in v.items():
        grad = got["d" + name][0]
        flat = t.view(-1)
        for i in range(0, flat.numel(), 5):
            keep = flat[i].item()
            flat[i] = keep + h
            up = loss(v)
            flat[i] = keep - h
            down = loss(v)
            flat[i] = keep
            assert abs((up - down) / (2 * h) - grad.reshape(-1)[i]) < 1e-7 * (1 + abs(up) / h * 1e-5)


def norm_cfg(**over):
    d = dict(T=4, first_row=0, p=0.0, H=64, dtype=N.MOE_BF16, param_dtype=N.MOE_F32,
             gate=N.MOE_GATE_NONE, eps=1e-6, residual_scale=1.0, branch_scale=1.0)
    d.update(over)
    return N.MoeNormCfg(**d)


FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first
FAKE2 = ctypes.c_void_p(1 << 21)
ODD = ctypes.c_void_p((1 << 20) + 8)
BAD_CFGS = [dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=12), dict(H=16392), dict(first_row=-1),
            dict(first_row=(1 << 32) - 3), dict(dtype=3), dict(dtype=-1),
            dict(param_dtype=N.MOE_F16), dict(gate=4), dict(gate=-1), dict(p=-0.1), dict(p=1.1),
            dict(p=float("nan")), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")),
            dict(residual_scale=float("inf")), dict(branch_scale=float("nan"))]


def fwd(lib, cfg, **over):
    p = dict(x=FAKE, y=FAKE, w_post=FAKE, gate=None, w_next=FAKE, rng=FAKE, row_ids=None, r=FAKE,
             n=FAKE2)
    p.update(over)
    return lib.moe_residual_norm(ctypes.byref(cfg), *p.values(), None)


def bwd(lib, cfg, ws_bytes=1 << 40, **over):
    p = dict(r=FAKE, y=FAKE, w_post=FAKE, gate=None, w_next=FAKE, rng=FAKE, row_ids=None, dr=FAKE,
             dn=FAKE, dx=FAKE, dy=FAKE2, dw_post=FAKE, dgate=None, dw_next=FAKE, ws=FAKE)
    p.update(over)
    return lib.moe_residual_norm_backward(ctypes.byref(cfg), *p.values(), ws_bytes, None)


@pytest.mark.parametrize("over", BAD_CFGS)
def test_bad_norm_configurations_rejected(lib, over):
    c = norm_cfg(**over)
    assert fwd(lib, c) == N.MOE_ERR_SHAPE
    assert bwd(lib, c) == N.MOE_ERR_SHAPE
    assert lib.moe_residual_norm_workspace_bytes(ctypes.byref(c)) == 0
    if not {"gate", "eps", "param_dtype", "residual_scale", "branch_scale"} & set(over):
        assert lib.moe_dropout(c.T, c.H, c.dtype, c.p, FAKE, FAKE, c.first_row, None, FAKE,
                               None) == N.MOE_ERR_SHAPE


def test_norm_pointer_combinations_rejected(lib):
    c = norm_cfg()
    for over in (dict(x=None), dict(r=None), dict(n=None), dict(w_next=None), dict(gate=FAKE),
                 dict(x=ODD), dict(y=ODD), dict(w_post=ODD), dict(w_next=ODD), dict(r=ODD),
                 dict(n=ODD), dict(y=None), dict(y=None, r=None), dict(n=FAKE)):
        assert fwd(lib, c, **over) == N.MOE_ERR_ARG, over
    for over in (dict(r=None), dict(dx=None), dict(dy=None), dict(dn=None), dict(dw_next=None),
                 dict(dw_post=None), dict(w_post=None), dict(w_next=None), dict(gate=FAKE),
                 dict(dgate=FAKE), dict(dx=ODD), dict(dr=ODD), dict(y=None), dict(dy=FAKE)):
        assert bwd(lib, c, **over) == N.MOE_ERR_ARG, over
    assert bwd(lib, c, w_next=None, dn=None, dw_next=None, dr=None) == N.MOE_ERR_ARG
    need = lib.moe_residual_norm_workspace_bytes(ctypes.byref(c))
    assert need > 0
    assert bwd(lib, c, ws_bytes=need - 1) == N.MOE_ERR_WORKSPACE
    assert bwd(lib, c, ws=None) == N.MOE_ERR_WORKSPACE
    g = norm_cfg(gate=N.MOE_GATE_FULL)
    assert fwd(lib, g) == N.MOE_ERR_ARG
    assert fwd(lib, g, gate=ODD) == N.MOE_ERR_ARG
    d = norm_cfg(p=0.5)
    assert fwd(lib, d, rng=None) == N.MOE_ERR_ARG
    assert bwd(lib, d, rng=None) == N.MOE_ERR_ARG
    assert fwd(lib, d, y=None, w_post=None, r=None) == N.MOE_ERR_ARG
    assert lib.moe_residual_norm(None, *[FAKE] * 9, None) == N.MOE_ERR_ARG
    assert fwd(lib, norm_cfg(T=0)) == N.MOE_OK  # a no-op
    for args in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None), (ODD, FAKE, FAKE),
                 (FAKE, FAKE, ODD)):
        x, rng, out = args
        assert lib.moe_dropout(4, 64, 0, 0.5, x, rng, 0, None, out, None) == N.MOE_ERR_ARG


def test_binding_refusals(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    bad = [lambda: moe.residual_norm(x.int(), x, w_next=w),
           lambda: moe.residual_norm(x[0], x, w_next=w),
           lambda: moe.residual_norm(x.t(), x.t(), w_next=w),
           lambda: moe.residual_norm(x, x.float(), w_next=w),
           lambda: moe.residual_norm(x, x, w_next=w[:32]),
           lambda: moe.residual_norm(x, x, w_next=w.double()),
           lambda: moe.residual_norm(x, x, w_next=w, w_post=w.bfloat16()),
           lambda: moe.residual_norm(x, x, gate=torch.ones(4), w_next=w),
           lambda: moe.residual_norm(x, x, gate=torch.ones(4, 64), w_next=w),
           lambda: moe.residual_norm(x, w_post=w, w_next=w),
           lambda: moe.residual_norm(x),
           lambda: moe.residual_norm(x, w_next=w, residual_scale=2.0),
           lambda: moe.residual_norm(x, x, p=0.5, w_next=w),
           lambda: moe.residual_norm(x, x, n=x),
           lambda: moe.residual_norm(x, w_next=w, r=x),
           lambda: moe.residual_norm(x, x, row_ids=torch.zeros(4), w_next=w),
           lambda: moe.residual_norm_backward(x, x, dr=x, dn=x),
           lambda: moe.residual_norm_backward(x, x, dr=x, w_next=w),
           lambda: moe.residual_norm_backward(x, x),
           lambda: moe.dropout(x, 0.5, None),
           lambda: moe.dropout(x, 0.5, torch.zeros(2)),
           lambda: moe.dropout(x, 0.5, torch.zeros(2, dtype=torch.int64)),  # not on a GPU
           lambda: moe.residual_norm(x, x, w_next=w)]
    for f in bad:
        with pytest.raises(moe.MoeError):
            f()


def test_rng_state_wraps():
    s = moe.rng_state(2 ** 64 - 1, 2 ** 63, device="cpu").tolist()
    assert s == [-1, -2 ** 63]
    assert moe.rng_state(5, 7, device="cpu").tolist() == [5, 7]


def test_binding_fails_loudly_when_it_is_not_built(lib, monkeypatch, tmp_path):
    monkeypatch.setattr(N, "BINDING_PATH", str(tmp_path / "missing.so"))
    monkeypatch.setattr(N, "_binding", None)
    with pytest.raises(RuntimeError, match="not built"):
        moe.dropout(torch.zeros(2, 8), 0.5, moe.rng_state(1, device="cpu"))


PLACES = """
#include <stdio.h>
#include "red_layout.cuh"
int main()
{
    int half, k, warp;
    printf("%d\\n", moe::kRedFloats<3>);
    while (scanf("%d %d %d", &half, &k, &warp) == 3)
        printf("%d\\n", moe::red_place<3>(half, k, warp));
}
"""


@pytest.mark.parametrize("sums", [(3, 2), (3,), (2,)])
def test_reductions_one_barrier_apart_do_not_meet(tmp_path, sums):
    """The backward's reductions over a row's warps, `sums` values each, row after row: between
    one call's reads and the next one's writes there is no barrier, so their places are disjoint;
    every place is inside the buffer and a call's places are its own."""
    (tmp_path / "places.cpp").write_text(PLACES)
    subprocess.run(["g++", "-std=c++17", "-x", "c++", str(tmp_path / "places.cpp"), "-I",
                    build.CSRC, "-o", str(tmp_path / "places")], check=True)
    calls = [(i & 1, k) for i, k in enumerate(sums * 6)]
    asked = [(h, k, w) for h, n in calls for k in range(n) for w in range(32)]
    out = subprocess.run([str(tmp_path / "places")], check=True, text=True, capture_output=True,
                         input="\n".join("%d %d %d" % a for a in asked)).stdout.split()
    floats, places = int(out[0]), iter(map(int, out[1:]))
    used = [[next(places) for _ in range(32 * n)] for _, n in calls]
    for i, u in enumerate(used):
        assert len(set(u)) == len(u) and min(u) >= 0 and max(u) < floats
        assert i == 0 or not set(u) & set(used[i - 1]), (i, sums)


def test_binding_of_another_torch_is_rebuilt_and_not_loaded(lib, monkeypatch):
    """The binding is compiled against torch's C++ headers: another version's is out of date for
    the build, and loading it is refused with what to do."""
    assert build._binding_up_to_date()
    monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    assert not build._binding_up_to_date()
    monkeypatch.setattr(N, "_binding", None)
    with pytest.raises(RuntimeError, match="other.*build"):
        moe.dropout(torch.zeros(2, 8), 0.5, moe.rng_state(1, device="cpu"))
    monkeypatch.undo()
    assert build._binding_up_to_date()
    with pytest.raises(moe.MoeError):  # loaded, and refuses the host's tensors
        moe.dropout(torch.zeros(2, 8), 0.5, moe.rng_state(1, device="cpu"))


def test_the_library_builds_without_torch(lib, monkeypatch, capsys):
    """The kernels' library needs nvcc alone, for whoever calls the C ABI: without torch the
    binding, which is torch's, is left out with a note."""
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    assert build.build() == build.LIB_PATH
    assert "without moe_binding.so" in capsys.readouterr().err
    monkeypatch.undo()
    assert build._binding_up_to_date()
