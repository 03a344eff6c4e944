"""Python binding of libmoe_b200: torch tensors in, the C ABI's calls out (through ctypes for the
layer's calls, through csrc/binding.cpp for the small ones around it).

Argument marshalling only -- shapes, dtypes and devices are checked, buffers are
allocated with torch (device memory is torch's), and every step of the layer runs in
the library's CUDA kernels on torch's current stream. Calls fail closed: a nonzero
return code raises ``MoeError``; with ``check=True`` the stream is synchronised and a
nonzero device status word (NaN scores, zero renormalisation denominator, bad expert
id, pipeline timeout) raises ``StatusError`` ("DSV4 Flash MoE Train-Inference
Consistency Roadmap", Follow-Up Issue Buckets: mismatches fail closed; UniRL PR #430:
abort rather than continue on a parity failure).
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional, Sequence

import torch

from . import _native as N

SOFTMAX = N.MOE_SOFTMAX
SIGMOID = N.MOE_SIGMOID
SQRTSOFTPLUS = N.MOE_SQRTSOFTPLUS
STATUS_NAMES = ("nan_tokens", "zero_denominator", "bad_expert_id", "pipeline_timeout",
                "bad_rows")


class MoeError(RuntimeError):
    pass


class StatusError(MoeError):
    def __init__(self, words):
        self.words = list(words)
        named = {n: w for n, w in zip(STATUS_NAMES, self.words) if w}
        super().__init__(f"device status reports anomalies: {named}")


@dataclasses.dataclass(frozen=True)
class Config:
    T: int
    H: int
    E: int
    K: int
    I: int
    I_shared: int = 0
    score_fn: int = SOFTMAX
    renorm: bool = True
    route_scale: float = 1.0
    n_group: int = 0        # group-limited selection, 0 = off
    topk_group: int = 0

    @classmethod
    def of(cls, shape, T: Optional[int] = None) -> "Config":
        """From a workload shape (anything with the same field names)."""
        return cls(T=shape.T if T is None else T, H=shape.H, E=shape.E, K=shape.K, I=shape.I,
                   I_shared=shape.I_shared, score_fn=shape.score_fn, renorm=bool(shape.renorm),
                   route_scale=float(shape.route_scale),
                   n_group=int(getattr(shape, "n_group", 0)),
                   topk_group=int(getattr(shape, "topk_group", 0)))

    def with_T(self, T: int) -> "Config":
        return dataclasses.replace(self, T=T)

    def c(self) -> N.MoeCfg:
        return N.MoeCfg(self.T, self.H, self.E, self.K, self.I, self.I_shared, self.score_fn,
                        int(bool(self.renorm)), float(self.route_scale), int(self.n_group),
                        int(self.topk_group))


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()  # an int, taken as a pointer by the signatures


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need(t, name, dtype, shape, dev):
    if t is not None and t.dtype is dtype and t.shape == shape and t.device == dev and \
            t.is_contiguous():
        return t
    if t is None:
        raise MoeError(f"{name} is required")
    if t.dtype != dtype:
        raise MoeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise MoeError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != dev:
        raise MoeError(f"{name}: on {t.device}, expected {dev}")
    if not t.is_contiguous():
        raise MoeError(f"{name} must be contiguous")
    return t


def _opt(t, name, dtype, shape, dev):
    return None if t is None else _need(t, name, dtype, shape, dev)


def _rc(code: int, what: str):
    if code != N.MOE_OK:
        raise MoeError(f"{what}: {N.status_string(code)} ({code})")


def workspace_bytes(cfg: Config, stage: int) -> int:
    return int(N.load().moe_workspace_bytes(ctypes.byref(cfg.c()), stage))


def new_status(dev) -> torch.Tensor:
    return torch.zeros(N.MOE_STATUS_WORDS, dtype=torch.int32, device=dev)


def _status(status: Optional[torch.Tensor], dev) -> torch.Tensor:
    """The given status words, checked, or new ones."""
    if status is None:
        return new_status(dev)
    if status.dtype != torch.int32 or status.device != dev or not status.is_contiguous() or \
            status.numel() < N.MOE_STATUS_WORDS:
        raise MoeError(f"status: {status.dtype} {tuple(status.shape)} on {status.device}, expected "
                       f"{N.MOE_STATUS_WORDS} contiguous torch.int32 words on {dev}")
    return status


def check_status(status: torch.Tensor, stream_sync: bool = True):
    if stream_sync:
        torch.cuda.current_stream(status.device).synchronize()
    words = status.cpu().tolist()
    if any(words):
        raise StatusError(words)


def _ws(nbytes: int, dev, ws: Optional[torch.Tensor]) -> torch.Tensor:
    """The given workspace, checked, or a new one."""
    if ws is not None:
        if ws.device != dev:
            raise MoeError(f"workspace on {ws.device}, expected {dev}")
        if not ws.is_contiguous():
            raise MoeError("the workspace must be contiguous")
        if ws.numel() * ws.element_size() < nbytes:
            raise MoeError(f"workspace of {ws.numel() * ws.element_size()} bytes < {nbytes}")
        return ws
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)


# ------------------------------------------------------------------ stages

def route(cfg: Config, x=None, w_router=None, logits=None, logit_bias=None, sel_bias=None,
          token_mask=None, status=None, check: bool = True):
    """Routing boundary. With x: logits are computed (returned); with x=None the given
    fp32 logits [T,E] are routed. Returns (logits, topk_ids, topk_w)."""
    dev = (x if x is not None else logits).device
    T, H, E, K = cfg.T, cfg.H, cfg.E, cfg.K
    if x is not None:
        _need(x, "x", torch.bfloat16, (T, H), dev)
        _need(w_router, "w_router", torch.bfloat16, (E, H), dev)
        logits = torch.empty(T, E, dtype=torch.float32, device=dev) if logits is None else logits
    _need(logits, "logits", torch.float32, (T, E), dev)
    _opt(logit_bias, "logit_bias", torch.float32, (E,), dev)
    _opt(sel_bias, "sel_bias", torch.float32, (E,), dev)
    _opt(token_mask, "token_mask", torch.uint8, (T,), dev)
    ids = torch.empty(T, K, dtype=torch.int32, device=dev)
    w = torch.empty(T, K, dtype=torch.float32, device=dev)
    st = _status(status, dev)
    _rc(N.load().moe_route(ctypes.byref(cfg.c()), _p(x), _p(w_router), _p(logit_bias),
                           _p(sel_bias), _p(token_mask), _p(logits), _p(ids), _p(w), _p(st),
                           _stream(dev)), "moe_route")
    if check:
        check_status(st)
    return logits, ids, w


def permute(cfg: Config, topk_ids, x=None, want_x_perm: bool = True, status=None,
            check: bool = True):
    """Dispatch boundary. Returns (offsets [E+1], perm_token [T*K], dest_row [T,K],
    x_perm [T*K,H] or None)."""
    dev = topk_ids.device
    T, K, E, H = cfg.T, cfg.K, cfg.E, cfg.H
    _need(topk_ids, "topk_ids", torch.int32, (T, K), dev)
    _opt(x, "x", torch.bfloat16, (T, H), dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm_token = torch.full((T * K,), -1, dtype=torch.int32, device=dev)
    dest_row = torch.empty(T, K, dtype=torch.int32, device=dev)
    x_perm = None
    if want_x_perm and x is not None:
        x_perm = torch.empty(T * K, H, dtype=torch.bfloat16, device=dev)
    nbytes = workspace_bytes(cfg, N.MOE_STAGE_PERMUTE)
    ws = _ws(nbytes, dev, None)
    st = _status(status, dev)
    _rc(N.load().moe_permute(ctypes.byref(cfg.c()), _p(topk_ids), _p(x), _p(offsets),
                             _p(perm_token), _p(dest_row), _p(x_perm), _p(st), _p(ws),
                             ws.numel(), _stream(dev)), "moe_permute")
    if check:
        check_status(st)
    return offsets, perm_token, dest_row, x_perm


def grouped_ffn(cfg: Config, x, x_perm, perm_token, offsets, w13, w2, w13_s=None, w2_s=None,
                status=None, check: bool = True):
    """Expert boundary. Returns (y [T*K,H], y_shared [T,H] or None)."""
    dev = offsets.device
    T, H, E, K, I, Is = cfg.T, cfg.H, cfg.E, cfg.K, cfg.I, cfg.I_shared
    _opt(x, "x", torch.bfloat16, (T, H), dev)
    _opt(x_perm, "x_perm", torch.bfloat16, (T * K, H), dev)
    _opt(perm_token, "perm_token", torch.int32, (T * K,), dev)
    _need(offsets, "offsets", torch.int32, (E + 1,), dev)
    _need(w13, "w13", torch.bfloat16, (E, 2 * I, H), dev)
    _need(w2, "w2", torch.bfloat16, (E, H, I), dev)
    if Is:
        _need(w13_s, "w13_s", torch.bfloat16, (2 * Is, H), dev)
        _need(w2_s, "w2_s", torch.bfloat16, (H, Is), dev)
    y = torch.empty(T * K, H, dtype=torch.bfloat16, device=dev)
    y_s = torch.empty(T, H, dtype=torch.bfloat16, device=dev) if Is else None
    ws = _ws(workspace_bytes(cfg, N.MOE_STAGE_FFN), dev, None)
    st = _status(status, dev)
    _rc(N.load().moe_grouped_ffn(ctypes.byref(cfg.c()), _p(x), _p(x_perm), _p(perm_token),
                                 _p(offsets), _p(w13), _p(w2), _p(w13_s), _p(w2_s), _p(y),
                                 _p(y_s), _p(st), _p(ws), ws.numel(), _stream(dev)),
        "moe_grouped_ffn")
    if check:
        check_status(st)
    return y, y_s


def combine(cfg: Config, y, topk_w, dest_row, y_shared=None, token_mask=None,
            order_invariant: bool = False):
    """Reduction boundary. Returns out [T,H] bf16. order_invariant=True runs the
    canonical-order variant (moe_combine_invariant) instead of the rank-order contract."""
    dev = y.device
    T, H, K = cfg.T, cfg.H, cfg.K
    if y.dim() != 2 or y.shape[1] != H or y.dtype != torch.bfloat16 or not y.is_contiguous():
        raise MoeError("y must be a contiguous bf16 [rows, H] tensor")
    _need(topk_w, "topk_w", torch.float32, (T, K), dev)
    _need(dest_row, "dest_row", torch.int32, (T, K), dev)
    _opt(y_shared, "y_shared", torch.bfloat16, (T, H), dev)
    _opt(token_mask, "token_mask", torch.uint8, (T,), dev)
    out = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    fn = N.load().moe_combine_invariant if order_invariant else N.load().moe_combine
    _rc(fn(ctypes.byref(cfg.c()), _p(y), _p(topk_w), _p(dest_row), _p(y_shared),
           _p(token_mask), _p(out), _stream(dev)), "moe_combine")
    return out


def pipeline_wait_selftest(dev, limit_cycles: int = 1_000_000, check: bool = True):
    """Run one bounded pipeline wait that nothing satisfies (moe_pipeline_wait_selftest):
    it gives up after limit_cycles and counts a pipeline timeout in the returned status
    words; with check=True the count raises StatusError, as in any other call."""
    st = new_status(dev)
    _rc(N.load().moe_pipeline_wait_selftest(_p(st), int(limit_cycles), _stream(st.device)),
        "moe_pipeline_wait_selftest")
    if check:
        check_status(st)
    return st


def router_stats(cfg: Config, logits, offsets, token_mask=None):
    """Router statistics of a routed batch: {tokens_per_expert [E] int32, mean_prob [E]
    fp32, aux [1] fp32} (the load-balance value E * sum_e load_e * mean_prob_e, K when
    balanced). logits and offsets as returned by route()/permute() or forward(keep=True)."""
    dev = logits.device
    T, E = cfg.T, cfg.E
    _need(logits, "logits", torch.float32, (T, E), dev)
    _need(offsets, "offsets", torch.int32, (E + 1,), dev)
    _opt(token_mask, "token_mask", torch.uint8, (T,), dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    mp = torch.empty(E, dtype=torch.float32, device=dev)
    aux = torch.empty(1, dtype=torch.float32, device=dev)
    ws = _ws(workspace_bytes(cfg, N.MOE_STAGE_STATS), dev, None)
    _rc(N.load().moe_router_stats(ctypes.byref(cfg.c()), _p(logits), _p(token_mask),
                                  _p(offsets), _p(counts), _p(mp), _p(aux), _p(ws), ws.numel(),
                                  _stream(dev)), "moe_router_stats")
    return {"tokens_per_expert": counts, "mean_prob": mp, "aux": aux}


# ------------------------------------------------------------------ around the layer

_DTYPES = {torch.bfloat16: N.MOE_BF16, torch.float16: N.MOE_F16, torch.float32: N.MOE_F32}


def _call(dev: torch.device, fn, *args):
    """fn(*args, stream) on dev's current stream, with dev the current device. (The raw calls:
    torch.cuda's own wrappers cost as much as the launch of a small kernel.)"""
    if dev.type != "cuda":
        raise MoeError(f"tensors on {dev}, expected a CUDA device")
    i = dev.index
    if i == torch._C._cuda_getDevice():
        return fn(*args, torch._C._cuda_getCurrentRawStream(i))
    with torch.cuda.device(dev):
        return fn(*args, torch._C._cuda_getCurrentRawStream(i))


def _native():
    """The native part of the binding."""
    return N._binding or N.load_binding(MoeError)


def _status_for(t):
    """Status words beside a tensor (None for what the call will refuse)."""
    return new_status(t.device) if isinstance(t, torch.Tensor) and t.is_cuda else None


def rng_state(seed: int, offset: int = 0, device="cuda") -> torch.Tensor:
    """The device state of the dropout masks, int64 (seed, offset): calls that share it share
    their masks. Change it (in place, under a captured graph) to draw new ones."""
    wrap = [(int(v) + 2 ** 63) % 2 ** 64 - 2 ** 63 for v in (seed, offset)]
    return torch.tensor(wrap, dtype=torch.int64, device=device)


def residual_norm(x, y=None, w_post=None, gate=None, w_next=None, eps: float = 1e-6,
                  residual_scale: float = 1.0, branch_scale: float = 1.0, p: float = 0.0,
                  rng=None, first_row: int = 0, row_ids=None, r=None, n=None):
    """What joins two blocks (moe_residual_norm), in one kernel:

        r = residual_scale * x + branch_scale * gate * dropout(rmsnorm(y) * w_post)
        n = rmsnorm(r) * w_next

    x, y [T,H] of one type (bf16, fp16, fp32); w_post, w_next [H] and gate ([H], [T,1] or
    [T,H]) optional; weights fp32 or of x's type, a [T,H] gate of x's type. y=None: the norm
    before the first block. p, rng, first_row, row_ids: see dropout. r, n: outputs to write
    (r may be x, n may be y). Returns (r, n), n None without w_next; r is x without y."""
    return _native().residual_norm(x, y, w_post, gate, w_next, eps, residual_scale, branch_scale,
                                   p, rng, first_row, row_ids, r, n)


def residual_norm_backward(r, y=None, dr=None, dn=None, w_post=None, gate=None, w_next=None,
                           eps: float = 1e-6, residual_scale: float = 1.0,
                           branch_scale: float = 1.0, p: float = 0.0, rng=None,
                           first_row: int = 0, row_ids=None) -> dict:
    """Gradients of sum(dr * r + dn * n) of residual_norm (moe_residual_norm_backward):
    {dx, dy, dw_post, dgate, dw_next}, those that exist. r is the forward's result (x where it
    had no y), the other arguments are the forward's; dn is given exactly with w_next, dr may
    be None. dx, dy and a [T,H] gate's gradient have r's type, the others are fp32. The norm
    statistics and the dropout mask are recomputed; nothing else is kept from the forward."""
    return _native().residual_norm_backward(r, y, dr, dn, w_post, gate, w_next, eps,
                                            residual_scale, branch_scale, p, rng, first_row,
                                            row_ids)


def dropout(x, p: float, rng, first_row: int = 0, row_ids=None, out=None):
    """Dropout of x [T,H] (bf16, fp16 or fp32) with a mask that is never stored (moe_dropout):
    out = x / P(keep) where kept, 0 elsewhere. The mask is a function of rng (rng_state()), the
    row and the column alone; row t is first_row + t, or row_ids[t], so a token keeps its mask
    in any batch. The gradient is dropout(dout) with the same p, rng and rows. out may be x."""
    return _native().dropout(x, p, rng, first_row, row_ids, out)


# ------------------------------------------------------------------ backward

def backward_workspace(cfg: Config, dev) -> torch.Tensor:
    """A workspace for forward_train() + backward(saved=True) (or backward alone)."""
    return _ws(workspace_bytes(cfg, N.MOE_STAGE_BACKWARD), dev, None)


def forward_train(cfg: Config, x, w_router, w13, w2, ws, logit_bias=None, sel_bias=None,
                  token_mask=None, w13_s=None, w2_s=None, status=None, check: bool = True):
    """The forward of a training step (moe_forward_train): the same output as forward(), and
    the intermediates the backward needs left in `ws` (backward_workspace()). Returns
    (out [T,H] bf16, {logits, topk_ids, topk_w}); then backward(..., ws=ws, saved=True)."""
    dev = x.device
    T, H, E, K, I, Is = cfg.T, cfg.H, cfg.E, cfg.K, cfg.I, cfg.I_shared
    _need(x, "x", torch.bfloat16, (T, H), dev)
    _need(w_router, "w_router", torch.bfloat16, (E, H), dev)
    _need(w13, "w13", torch.bfloat16, (E, 2 * I, H), dev)
    _need(w2, "w2", torch.bfloat16, (E, H, I), dev)
    _opt(logit_bias, "logit_bias", torch.float32, (E,), dev)
    _opt(sel_bias, "sel_bias", torch.float32, (E,), dev)
    _opt(token_mask, "token_mask", torch.uint8, (T,), dev)
    if Is:
        _need(w13_s, "w13_s", torch.bfloat16, (2 * Is, H), dev)
        _need(w2_s, "w2_s", torch.bfloat16, (H, Is), dev)
    out = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    b = {"logits": torch.empty(T, E, dtype=torch.float32, device=dev),
         "topk_ids": torch.empty(T, K, dtype=torch.int32, device=dev),
         "topk_w": torch.empty(T, K, dtype=torch.float32, device=dev)}
    nbytes = workspace_bytes(cfg, N.MOE_STAGE_BACKWARD)
    ws = _ws(nbytes, dev, ws)
    st = _status(status, dev)
    _rc(N.load().moe_forward_train(ctypes.byref(cfg.c()), _p(x), _p(w_router), _p(logit_bias),
                                   _p(sel_bias), _p(token_mask), _p(w13), _p(w2), _p(w13_s),
                                   _p(w2_s), _p(out), _p(b["logits"]), _p(b["topk_ids"]),
                                   _p(b["topk_w"]), _p(st), _p(ws), nbytes, _stream(dev)),
        "moe_forward_train")
    if check:
        check_status(st)
    return out, b


def backward(cfg: Config, x, w_router, w13, w2, logits, topk_ids, topk_w, dout, token_mask=None,
             w13_s=None, w2_s=None, ws=None, status=None, keep: bool = False,
             saved: bool = False, check: bool = True) -> dict:
    """Gradients of sum(dout * out) of the layer for the forward's routes (moe_backward):
    {dx [T,H] bf16, dw_router [E,H], dw13 [E,2I,H], dw2 [E,H,I] fp32 (+ dw13_s, dw2_s with a
    shared expert)}; keep=True adds d_topk_w [T,K] and dlogits [T,E] (fp32).
    logits, topk_ids, topk_w: as forward(keep=True) or forward_train() returned them.
    saved=True: ws holds forward_train()'s intermediates for the same inputs (no recompute)."""
    if saved and ws is None:
        raise MoeError("saved=True needs the workspace forward_train() wrote")
    dev = x.device
    T, H, E, K, I, Is = cfg.T, cfg.H, cfg.E, cfg.K, cfg.I, cfg.I_shared
    _need(x, "x", torch.bfloat16, (T, H), dev)
    _need(w_router, "w_router", torch.bfloat16, (E, H), dev)
    _need(w13, "w13", torch.bfloat16, (E, 2 * I, H), dev)
    _need(w2, "w2", torch.bfloat16, (E, H, I), dev)
    _need(logits, "logits", torch.float32, (T, E), dev)
    _need(topk_ids, "topk_ids", torch.int32, (T, K), dev)
    _need(topk_w, "topk_w", torch.float32, (T, K), dev)
    _need(dout, "dout", torch.bfloat16, (T, H), dev)
    _opt(token_mask, "token_mask", torch.uint8, (T,), dev)
    if Is:
        _need(w13_s, "w13_s", torch.bfloat16, (2 * Is, H), dev)
        _need(w2_s, "w2_s", torch.bfloat16, (H, Is), dev)
    g = {"dx": torch.empty(T, H, dtype=torch.bfloat16, device=dev),
         "dw_router": torch.empty(E, H, dtype=torch.float32, device=dev),
         "dw13": torch.empty(E, 2 * I, H, dtype=torch.float32, device=dev),
         "dw2": torch.empty(E, H, I, dtype=torch.float32, device=dev),
         "dw13_s": torch.empty(2 * Is, H, dtype=torch.float32, device=dev) if Is else None,
         "dw2_s": torch.empty(H, Is, dtype=torch.float32, device=dev) if Is else None}
    if keep:
        g["d_topk_w"] = torch.empty(T, K, dtype=torch.float32, device=dev)
        g["dlogits"] = torch.empty(T, E, dtype=torch.float32, device=dev)
    nbytes = workspace_bytes(cfg, N.MOE_STAGE_BACKWARD)
    ws = _ws(nbytes, dev, ws)
    st = _status(status, dev)
    _rc(N.load().moe_backward(ctypes.byref(cfg.c()), _p(x), _p(w_router), _p(token_mask),
                              _p(w13), _p(w2), _p(w13_s), _p(w2_s), _p(logits), _p(topk_ids),
                              _p(topk_w), _p(dout), _p(g["dx"]), _p(g["dw_router"]),
                              _p(g["dw13"]), _p(g["dw2"]), _p(g["dw13_s"]), _p(g["dw2_s"]),
                              _p(g.get("d_topk_w")), _p(g.get("dlogits")), int(bool(saved)),
                              _p(st), _p(ws), nbytes, _stream(dev)), "moe_backward")
    if check:
        check_status(st)
    return g


# ------------------------------------------------------------------ whole layer

def forward(cfg: Config, x, w_router, w13, w2, logit_bias=None, sel_bias=None, token_mask=None,
            w13_s=None, w2_s=None, out=None, ws=None, status=None, keep: bool = False,
            stage_events: Optional[Sequence] = None, check: bool = True):
    """The MoE layer (routing -> dispatch -> experts -> combine) in one C-ABI call.

    keep=True also returns the boundary tensors {logits, topk_ids, topk_w, offsets}.
    stage_events: MOE_NUM_STAGE_EVENTS torch.cuda.Event(enable_timing=True) recorded at
    the stage boundaries (for timing)."""
    dev = x.device
    T, H, E, K, I, Is = cfg.T, cfg.H, cfg.E, cfg.K, cfg.I, cfg.I_shared
    _need(x, "x", torch.bfloat16, (T, H), dev)
    _need(w_router, "w_router", torch.bfloat16, (E, H), dev)
    _need(w13, "w13", torch.bfloat16, (E, 2 * I, H), dev)
    _need(w2, "w2", torch.bfloat16, (E, H, I), dev)
    _opt(logit_bias, "logit_bias", torch.float32, (E,), dev)
    _opt(sel_bias, "sel_bias", torch.float32, (E,), dev)
    _opt(token_mask, "token_mask", torch.uint8, (T,), dev)
    if Is:
        _need(w13_s, "w13_s", torch.bfloat16, (2 * Is, H), dev)
        _need(w2_s, "w2_s", torch.bfloat16, (H, Is), dev)
    out = torch.empty(T, H, dtype=torch.bfloat16, device=dev) if out is None else out
    _need(out, "out", torch.bfloat16, (T, H), dev)
    ws = _ws(workspace_bytes(cfg, N.MOE_STAGE_FORWARD), dev, ws)
    st = _status(status, dev)
    b = {}
    if keep:
        b = {"logits": torch.empty(T, E, dtype=torch.float32, device=dev),
             "topk_ids": torch.empty(T, K, dtype=torch.int32, device=dev),
             "topk_w": torch.empty(T, K, dtype=torch.float32, device=dev),
             "offsets": torch.empty(E + 1, dtype=torch.int32, device=dev)}
    ev = None
    if stage_events is not None:
        if len(stage_events) != N.MOE_NUM_STAGE_EVENTS:
            raise MoeError(f"stage_events needs {N.MOE_NUM_STAGE_EVENTS} events")
        stream = torch.cuda.current_stream(dev)
        for e in stage_events:
            if e is not None and not e.cuda_event:
                e.record(stream)  # torch creates its events lazily, on first record
        ev = (ctypes.c_void_p * N.MOE_NUM_STAGE_EVENTS)(
            *[None if e is None else e.cuda_event for e in stage_events])
    _rc(N.load().moe_forward(ctypes.byref(cfg.c()), _p(x), _p(w_router), _p(logit_bias),
                             _p(sel_bias), _p(token_mask), _p(w13), _p(w2), _p(w13_s),
                             _p(w2_s), _p(out), _p(b.get("logits")), _p(b.get("topk_ids")),
                             _p(b.get("topk_w")), _p(b.get("offsets")), _p(st), _p(ws),
                             ws.numel(), ev, _stream(dev)), "moe_forward")
    if check:
        check_status(st)
    return (out, b) if keep else out


def forward_host_workspace_bytes(cfg: Config, chunk: int) -> int:
    return int(N.load().moe_forward_host_workspace_bytes(ctypes.byref(cfg.c()), int(chunk)))


def forward_host(cfg: Config, x_host, w_router, w13, w2, logit_bias=None, sel_bias=None,
                 token_mask=None, w13_s=None, w2_s=None, out_host=None, chunk: int = 6144,
                 ws=None, status=None, check: bool = True):
    """The layer from and to host memory in one C-ABI call, transfers overlapped with the
    compute in chunks around `chunk` tokens (half-size first and last chunks, middle ones of
    at most 1.5 x chunk; see moe_forward_host). x_host / out_host are CPU bf16 tensors (pin
    them for the overlap); weights, biases and the mask are on the device."""
    dev = w13.device
    T, H, E, K, I, Is = cfg.T, cfg.H, cfg.E, cfg.K, cfg.I, cfg.I_shared
    cpu = torch.device("cpu")
    _need(x_host, "x_host", torch.bfloat16, (T, H), cpu)
    out_host = torch.empty(T, H, dtype=torch.bfloat16).pin_memory() if out_host is None \
        else out_host
    _need(out_host, "out_host", torch.bfloat16, (T, H), cpu)
    _need(w_router, "w_router", torch.bfloat16, (E, H), dev)
    _need(w13, "w13", torch.bfloat16, (E, 2 * I, H), dev)
    _need(w2, "w2", torch.bfloat16, (E, H, I), dev)
    _opt(logit_bias, "logit_bias", torch.float32, (E,), dev)
    _opt(sel_bias, "sel_bias", torch.float32, (E,), dev)
    _opt(token_mask, "token_mask", torch.uint8, (T,), dev)
    if Is:
        _need(w13_s, "w13_s", torch.bfloat16, (2 * Is, H), dev)
        _need(w2_s, "w2_s", torch.bfloat16, (H, Is), dev)
    ws = _ws(forward_host_workspace_bytes(cfg, chunk), dev, ws)
    st = _status(status, dev)
    _rc(N.load().moe_forward_host(ctypes.byref(cfg.c()), _p(x_host), _p(w_router),
                                  _p(logit_bias), _p(sel_bias), _p(token_mask), _p(w13), _p(w2),
                                  _p(w13_s), _p(w2_s), _p(out_host), _p(st), int(chunk), _p(ws),
                                  ws.numel(), _stream(dev)), "moe_forward_host")
    if check:
        check_status(st)
    return out_host


# ------------------------------------------------------------------ experts in 4 bits

def mx_quantize(x, tiled: bool = True):
    """Rows of x [R,K] (bf16, fp16 or fp32, K a multiple of 32) in the microscaled 4-bit format
    (moe_mx_quantize): (codes [R,K/2], scales), both uint8. The scales are in the tensor core's
    tiles, [ceil(R/128), ceil(K/128), 512], as the products take them, or with tiled=False
    row-major, [R,K/32]."""
    return _native().mx_quantize(x, tiled)


def mx_weight(w):
    """Expert weights [E,N,K] (or one matrix [N,K]; N and K multiples of 128) in the microscaled
    4-bit format, as the products take them: (codes [E,N,K/2], scales in the tensor core's tiles
    [E,N/128,K/128,512]), both uint8."""
    if w.dim() not in (2, 3) or w.dtype not in _DTYPES or not w.is_contiguous():
        raise MoeError(f"w: a contiguous [E,N,K] or [N,K] bf16, fp16 or fp32 tensor is expected, "
                       f"got {w.dtype} {tuple(w.shape)}")
    *lead, n, k = w.shape
    if n % 128 or k % 128:
        raise MoeError(f"w: N and K must be multiples of 128, got {n} and {k}")
    dev = w.device
    codes = torch.empty(*lead, n, k // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(*lead, n // 128, k // 128, 512, dtype=torch.uint8, device=dev)
    rows = w.numel() // k if k else 0
    _rc(_call(dev, N.load().moe_mx_quantize, rows, k, _DTYPES[w.dtype], 1, _p(w), _p(codes),
              _p(scales)), "moe_mx_quantize")
    return codes, scales


def mx_dequantize(codes, scales, dtype=torch.bfloat16):
    """The values of mx_quantize's codes [R,K/2] and scales (in tiles, or row-major [R,K/32]),
    rounded to dtype: [R,K]."""
    return _native().mx_dequantize(codes, scales, dtype)


def _mx_need(w, name, n, k, dev, lead=()):
    """4-bit weights (codes, tiled scales) of matrices [n, k], lead = (how many,) or ()."""
    if w is None or len(w) != 2:
        raise MoeError(f"{name}: (codes, scales) of mx_weight() are expected")
    codes, scales = w  # once: a sequence may make its members when asked
    return (_need(codes, f"{name} codes", torch.uint8, lead + (n, k // 2), dev),
            _need(scales, f"{name} scales", torch.uint8, lead + (n // 128, k // 128, 512), dev))


def mx_grouped_gemm(codes, scales, offsets, w_codes, w_scales, swiglu: bool = False, out=None,
                    status=None, check: bool = True):
    """Rows in 4 bits (mx_quantize, scales in tiles), grouped by offsets [E+1], times 4-bit weights
    (mx_weight of [E,N,K]): [R,N] bf16, or with swiglu silu(first N/2 columns) * last N/2, [R,N/2]
    (moe_mx_grouped_gemm). Rows outside every group are left as they were in out."""
    if check and status is None:
        status = _status_for(codes)
    out = _native().mx_grouped_gemm(codes, scales, offsets, w_codes, w_scales, swiglu, out, status)
    if check:
        check_status(status)
    return out


def _mx_experts(cfg, w13, w2, w13_s, w2_s, dev):
    """The tensors of a layer's 4-bit expert weights, checked, in the order of the C ABI."""
    H, I, Is, E = cfg.H, cfg.I, cfg.I_shared, (cfg.E,)
    w = _mx_need(w13, "w13", 2 * I, H, dev, E) + _mx_need(w2, "w2", H, I, dev, E)
    if not Is:
        return w + (None, None, None, None)
    return w + _mx_need(w13_s, "w13_s", 2 * Is, H, dev) + _mx_need(w2_s, "w2_s", H, Is, dev)


def mx_grouped_ffn(cfg: Config, x, dest_row, offsets, w13, w2, w13_s=None, w2_s=None, ws=None,
                   status=None, check: bool = True):
    """The expert boundary with 4-bit experts (moe_mx_grouped_ffn): w13, w2 (and the shared
    expert's) as mx_weight() returned them, dest_row and offsets from permute(). Returns
    (y [T*K,H], y_shared [T,H] or None)."""
    if check and status is None:
        status = _status_for(x)
    y = _native().mx_grouped_ffn(cfg, x, dest_row, offsets, w13, w2, w13_s, w2_s, ws, status)
    if check:
        check_status(status)
    return y


def mx_forward(cfg: Config, x, w_router, w13, w2, logit_bias=None, sel_bias=None, token_mask=None,
               w13_s=None, w2_s=None, out=None, ws=None, status=None, keep: bool = False,
               check: bool = True):
    """The MoE layer with 4-bit experts in one call (moe_mx_forward): as forward(), with w13, w2
    (and the shared expert's) as mx_weight() returned them; the router stays bf16."""
    dev = x.device
    T, H, E, K = cfg.T, cfg.H, cfg.E, cfg.K
    _need(x, "x", torch.bfloat16, (T, H), dev)
    _need(w_router, "w_router", torch.bfloat16, (E, H), dev)
    w = _mx_experts(cfg, w13, w2, w13_s, w2_s, dev)
    _opt(logit_bias, "logit_bias", torch.float32, (E,), dev)
    _opt(sel_bias, "sel_bias", torch.float32, (E,), dev)
    _opt(token_mask, "token_mask", torch.uint8, (T,), dev)
    out = torch.empty(T, H, dtype=torch.bfloat16, device=dev) if out is None else out
    _need(out, "out", torch.bfloat16, (T, H), dev)
    lib, ref = N.load(), ctypes.byref(cfg.c())
    nbytes = lib.moe_workspace_bytes(ref, N.MOE_STAGE_MX_FORWARD)
    ws = _ws(nbytes, dev, ws)
    st = _status(status, dev)
    b = {}
    if keep:
        b = {"logits": torch.empty(T, E, dtype=torch.float32, device=dev),
             "topk_ids": torch.empty(T, K, dtype=torch.int32, device=dev),
             "topk_w": torch.empty(T, K, dtype=torch.float32, device=dev),
             "offsets": torch.empty(E + 1, dtype=torch.int32, device=dev)}
    _rc(_call(dev, lib.moe_mx_forward, ref, _p(x), _p(w_router),
              _p(logit_bias), _p(sel_bias), _p(token_mask), *map(_p, w), _p(out),
              _p(b.get("logits")), _p(b.get("topk_ids")), _p(b.get("topk_w")),
              _p(b.get("offsets")), _p(st), _p(ws), nbytes), "moe_mx_forward")
    if check:
        check_status(st)
    return (out, b) if keep else out


class MoELayer:
    """A layer holding its weights and a reusable workspace sized for up to max_T tokens.

    weights: dict with w_router, w13, w2 and optionally logit_bias, sel_bias, w13_s, w2_s
    (the layout of include/moe.h). Expert weights given as mx_weight() returned them make a
    layer with 4-bit experts (mx_forward); quantized() makes one from a bf16 layer."""

    def __init__(self, cfg: Config, weights: dict, max_T: Optional[int] = None):
        self.cfg = cfg
        self.w = weights
        self.max_T = cfg.T if max_T is None else max_T
        self.mx = not isinstance(weights["w13"], torch.Tensor)
        dev = (weights["w13"][0] if self.mx else weights["w13"]).device
        stage = N.MOE_STAGE_MX_FORWARD if self.mx else N.MOE_STAGE_FORWARD
        self.ws = _ws(workspace_bytes(cfg.with_T(self.max_T), stage), dev, None)
        self.status = new_status(dev)

    def quantized(self) -> "MoELayer":
        """The same layer with its experts in the microscaled 4-bit format."""
        if self.mx:
            return self
        w = {k: mx_weight(v) if k in ("w13", "w2", "w13_s", "w2_s") and v is not None else v
             for k, v in self.w.items()}
        return MoELayer(self.cfg, w, self.max_T)

    def forward_host(self, x_host, out_host=None, chunk: int = 6144, token_mask=None,
                     check=True):
        """The layer from pinned host memory to pinned host memory (see forward_host)."""
        if self.mx:
            raise MoeError("forward_host takes bf16 experts")
        T = x_host.shape[0]
        need = forward_host_workspace_bytes(self.cfg.with_T(T), chunk)
        if getattr(self, "_host_ws", None) is None or self._host_ws.numel() < need:
            self._host_ws = _ws(need, self.ws.device, None)
        w = self.w
        return forward_host(self.cfg.with_T(T), x_host, w["w_router"], w["w13"], w["w2"],
                            logit_bias=w.get("logit_bias"), sel_bias=w.get("sel_bias"),
                            token_mask=token_mask, w13_s=w.get("w13_s"), w2_s=w.get("w2_s"),
                            out_host=out_host, chunk=chunk, ws=self._host_ws,
                            status=self.status, check=check)

    def __call__(self, x, token_mask=None, out=None, keep=False, check=True, stage_events=None):
        T = x.shape[0]
        if T > self.max_T:
            raise MoeError(f"{T} tokens > the layer's max_T {self.max_T}")
        w = self.w
        if self.mx:
            if stage_events is not None:
                raise MoeError("stage events are recorded by a layer with bf16 experts")
            return mx_forward(self.cfg.with_T(T), x, w["w_router"], w["w13"], w["w2"],
                              logit_bias=w.get("logit_bias"), sel_bias=w.get("sel_bias"),
                              token_mask=token_mask, w13_s=w.get("w13_s"), w2_s=w.get("w2_s"),
                              out=out, ws=self.ws, status=self.status, keep=keep, check=check)
        return forward(self.cfg.with_T(T), x, w["w_router"], w["w13"], w["w2"],
                       logit_bias=w.get("logit_bias"), sel_bias=w.get("sel_bias"),
                       token_mask=token_mask, w13_s=w.get("w13_s"), w2_s=w.get("w2_s"),
                       out=out, ws=self.ws, status=self.status, keep=keep, check=check,
                       stage_events=stage_events)


class MoEBlock:
    """A layer and what joins its block to the next one:

        y = layer(n),  r = residual_scale * x + branch_scale * gate * dropout(rmsnorm(y) * w_post)
        n' = rmsnorm(r) * w_next

    x is the residual stream, n its norm under this block's weight -- the n' that the block
    before returned, or residual_norm(x, w_next=...)[1] before the first one. w_post, gate ([H])
    and w_next are optional; p is the dropout probability of the training forward (a plain call
    drops nothing). rng, first_row and row_ids: see dropout(). A training forward's ws belongs to
    it until its backward: blocks, or steps, in flight at once need one each. So does a layer's own
    workspace with calls or captured graphs that may run at the same time: a layer object each."""

    def __init__(self, layer: MoELayer, w_post=None, gate=None, w_next=None, eps: float = 1e-6,
                 residual_scale: float = 1.0, branch_scale: float = 1.0, p: float = 0.0):
        self.layer = layer
        self.p = p
        self.kw = dict(w_post=w_post, gate=gate, w_next=w_next, eps=eps,
                       residual_scale=residual_scale, branch_scale=branch_scale)

    def __call__(self, x, n, token_mask=None, check=True):
        """(r, n') for serving, with bf16 or 4-bit experts."""
        y = self.layer(n, token_mask=token_mask, check=check)
        return residual_norm(x, y, **self.kw)

    def forward_train(self, x, n, ws, rng=None, token_mask=None, first_row: int = 0, row_ids=None,
                      check=True):
        """(r, n', saved): the training forward, the layer's intermediates left in ws
        (backward_workspace()), what backward() needs besides in saved."""
        if self.layer.mx:
            raise MoeError("training needs bf16 experts")
        w, cfg = self.layer.w, self.layer.cfg.with_T(x.shape[0])
        y, b = forward_train(cfg, n, w["w_router"], w["w13"], w["w2"], ws,
                             logit_bias=w.get("logit_bias"), sel_bias=w.get("sel_bias"),
                             token_mask=token_mask, w13_s=w.get("w13_s"), w2_s=w.get("w2_s"),
                             check=check)
        drop = dict(p=self.p, rng=rng, first_row=first_row, row_ids=row_ids)
        r, n2 = residual_norm(x, y, **self.kw, **drop)
        return r, n2, dict(n=n, y=y, r=r, routes=b, ws=ws, token_mask=token_mask, drop=drop)

    def backward(self, saved: dict, dr=None, dn=None, check=True) -> dict:
        """Gradients of sum(dr * r + dn * n'): {dx, dn} of the inputs -- the dr and dn of the
        block before -- {dw_post, dgate, dw_next} as the block has them, and the layer's under
        "layer" (see backward(); its dx is this dn)."""
        w, cfg = self.layer.w, self.layer.cfg.with_T(saved["n"].shape[0])
        g = residual_norm_backward(saved["r"], saved["y"], dr=dr, dn=dn, **self.kw,
                                   **saved["drop"])
        b = saved["routes"]
        lay = backward(cfg, saved["n"], w["w_router"], w["w13"], w["w2"], b["logits"],
                       b["topk_ids"], b["topk_w"], g.pop("dy"), token_mask=saved["token_mask"],
                       w13_s=w.get("w13_s"), w2_s=w.get("w2_s"), ws=saved["ws"], saved=True,
                       check=check)
        g["dn"] = lay.pop("dx")
        g["layer"] = lay
        return g
