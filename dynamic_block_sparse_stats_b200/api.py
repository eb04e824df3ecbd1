"""Torch-facing wrapper of the Prism C ABI.

PyTorch provides device memory and the current stream; every computation runs
in libprism.so.  Tensors follow the layout of include/prism.h:
Q, K, V, O, dO bf16 [N, heads, head_dim] contiguous on one CUDA device, the
A2V norm map fp32 [N].

Calls take a torch.cuda.Stream as `stream` (default: the current one).  The
caller orders it behind whatever made the inputs, and keeps the inputs until it
is done.  What the call allocates, its workspace included, is that stream's
memory, and is not given out again before the current stream is done with it
too.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import math
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import PrismCkpt8, PrismLinear, PrismParams, PrismPlan, PrismSelect, check


# guidance bits and density modes of the ablation variants (include/prism.h)
GUIDE_NO_VIDEO, GUIDE_NO_A2V = 1, 2
DENSITY_BOTH, DENSITY_SPATIAL, DENSITY_TEMPORAL, DENSITY_A2V = 0, 1, 2, 3


def params(T, H, W, heads, head_dim, topk_frac=0.0, topk_abs=0, top_p=0.9, tau128=0.5, tau256=0.25,
           eps=1e-6, sm_scale=0.0, map_exponent=0.0, guidance=0, density=0) -> PrismParams:
    """Layer parameters; map_exponent 0 means the Lagrange value 1/2, and
    guidance = density = 0 is the method as published."""
    return PrismParams(T, H, W, heads, head_dim, tau128, tau256, eps, topk_frac, topk_abs, top_p, sm_scale,
                       map_exponent, guidance, density)


def params_for(w, **over) -> PrismParams:
    """Parameters of a synthetic workload (dynamic_block_sparse_stats_b200.synth.Workload)."""
    kw = dict(topk_frac=w.topk_frac, topk_abs=w.topk_abs, top_p=w.top_p)
    kw.update(over)
    return params(w.T, w.H, w.W, w.heads, w.head_dim, **kw)


def _stream(stream, device) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


_HERE = contextlib.nullcontext()


def _alloc_on(stream, dev):
    """Where a call's new tensors come from: with an explicit stream, from that
    stream's memory.  Memory of the current stream may still be in use there when
    the other stream writes it, and is given out again while that stream runs."""
    if not isinstance(stream, torch.cuda.Stream):
        return _HERE
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.stream(stream)


def _hand_over(stream, dev, *made):
    """New outputs of a call with an explicit stream: their memory waits for the
    caller's current stream too before it is given out again."""
    if isinstance(stream, torch.cuda.Stream):
        here = torch.cuda.current_stream(dev)
        if here != stream:
            for t in made:
                if t is not None:
                    t.record_stream(here)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _check_tensor(t, name, dtype, shape):
    """Structure of one tensor argument: type, dtype, shape, contiguity.  The
    C ABI sees bare pointers, so buffer sizes can only be checked here."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_workspace(ws, name):
    if not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8 or ws.dim() != 1 or not ws.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D uint8 tensor")


def _check_devices(named) -> torch.device:
    """Every (name, tensor) pair, None entries skipped, must live on one CUDA
    device; returns it.  Run after the structural checks, so that a wrong
    size is reported before a wrong device."""
    dev = None
    for name, t in named:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other arguments on {dev}")
    return dev


def _grid(p: PrismParams):
    return (p.T, p.H, p.W, p.heads, p.head_dim)


def _check_grid(p: PrismParams, q: PrismParams, what: str):
    if _grid(p) != _grid(q):
        raise ValueError(f"{what} was made for (T, H, W, heads, head_dim) = {_grid(q)}, "
                         f"the call is for {_grid(p)}")


def _sizes(p: PrismParams):
    N = p.T * p.H * p.W
    return N, (p.T // 8) * (p.H // 8) * (p.W // 8), N // 64


def _workspace(nbytes, device):
    # 256-byte alignment is guaranteed by the CUDA caching allocator
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def a2v_norm(hhat: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """prism_a2v_norm: ||h_hat||_2 of every row of the bf16 bridge output
    h_hat [N, width] (rows may be strided; width a multiple of 8) -> fp32 [N],
    the a2v_norm input of the next layer's plan."""
    if not isinstance(hhat, torch.Tensor) or hhat.dtype != torch.bfloat16 or hhat.dim() != 2:
        raise ValueError("hhat must be a 2-D bf16 tensor [N, width]")
    if hhat.stride(1) != 1:
        raise ValueError("hhat rows must be contiguous")
    n, width = hhat.shape
    if out is not None:
        _check_tensor(out, "a2v_norm", torch.float32, (n,))
    dev = _check_devices([("hhat", hhat), ("a2v_norm", out)])
    ld = hhat.stride(0) if n > 1 else width
    made = out is None
    with torch.cuda.device(dev), _alloc_on(stream, dev):
        out = out if out is not None else torch.empty((n,), dtype=torch.float32, device=dev)
        check(_lib.load().prism_a2v_norm(_ptr(hhat), n, width, ld, _ptr(out), _stream(stream, dev)))
    _hand_over(stream, dev, out if made else None)
    return out


@dataclass
class Plan:
    """Output of prism_plan (device tensors, Z zones, NB = N/64):
    zone_shape u8 [heads, Z] candidate id per zone; zone_g f64 [heads, Z, 3]
    (g_T, g_H, g_W); zone_rho f64 [heads, Z] normalised density; n_blocks
    i32 [heads]; blocks i32 [heads, NB, 4] {first permuted position, volume,
    natural index of the block's origin token, candidate id} (rows past
    n_blocks unspecified); perm / inv_perm i32 [heads, N]; ws the call's
    workspace."""
    p: PrismParams
    zone_shape: torch.Tensor
    zone_g: torch.Tensor
    zone_rho: torch.Tensor
    n_blocks: torch.Tensor
    blocks: torch.Tensor
    perm: torch.Tensor
    inv_perm: torch.Tensor
    ws: torch.Tensor

    def tensors(self):
        return (self.zone_shape, self.zone_g, self.zone_rho, self.n_blocks, self.blocks, self.perm, self.inv_perm, self.ws)

    def c_struct(self) -> PrismPlan:
        return PrismPlan(self.zone_shape.data_ptr(), self.zone_g.data_ptr(), self.zone_rho.data_ptr(),
                         self.n_blocks.data_ptr(), self.blocks.data_ptr(), self.perm.data_ptr(),
                         self.inv_perm.data_ptr())


def alloc_plan(p: PrismParams, device) -> Plan:
    N, Z, NB = _sizes(p)
    lib = _lib.load()
    ws = _workspace(lib.prism_plan_workspace_size(C.byref(p)), device)
    return Plan(p, torch.empty((p.heads, Z), dtype=torch.uint8, device=device),
                torch.empty((p.heads, Z, 3), dtype=torch.float64, device=device),
                torch.empty((p.heads, Z), dtype=torch.float64, device=device),
                torch.empty((p.heads,), dtype=torch.int32, device=device),
                torch.empty((p.heads, NB, 4), dtype=torch.int32, device=device),
                torch.empty((p.heads, N), dtype=torch.int32, device=device),
                torch.empty((p.heads, N), dtype=torch.int32, device=device), ws)


def _check_plan(p: PrismParams, pl: Plan):
    """Structural checks of a plan against the call's grid; returns its
    named tensors for the device check."""
    if not isinstance(pl, Plan):
        raise TypeError(f"plan must be an api.Plan, got {type(pl).__name__}")
    _check_grid(p, pl.p, "the plan")
    N, Z, NB = _sizes(p)
    h = p.heads
    named = []
    for name, dtype, shape in (("zone_shape", torch.uint8, (h, Z)), ("zone_g", torch.float64, (h, Z, 3)),
                               ("zone_rho", torch.float64, (h, Z)), ("n_blocks", torch.int32, (h,)),
                               ("blocks", torch.int32, (h, NB, 4)), ("perm", torch.int32, (h, N)),
                               ("inv_perm", torch.int32, (h, N))):
        _check_tensor(getattr(pl, name), "plan." + name, dtype, shape)
        named.append(("plan." + name, getattr(pl, name)))
    _check_workspace(pl.ws, "plan.ws")
    return named + [("plan.ws", pl.ws)]


def plan(p: PrismParams, V: torch.Tensor, a: torch.Tensor | None = None, out: Plan | None = None,
         stream=None) -> Plan:
    """prism_plan: zone statistics -> volumes, shapes, block table, permutation."""
    N = p.T * p.H * p.W
    _check_tensor(V, "V", torch.bfloat16, (N, p.heads, p.head_dim))
    if a is not None:
        _check_tensor(a, "a2v_norm", torch.float32, (N,))
    named = [("V", V), ("a2v_norm", a)] + (_check_plan(p, out) if out is not None else [])
    dev = _check_devices(named)
    made = out is None
    with torch.cuda.device(dev), _alloc_on(stream, dev):
        out = out if out is not None else alloc_plan(p, dev)
        cs = out.c_struct()
        check(_lib.load().prism_plan(C.byref(p), _ptr(V), _ptr(a), C.byref(cs), _ptr(out.ws), out.ws.numel(),
                                     _stream(stream, dev)))
    _hand_over(stream, dev, *(out.tensors() if made else ()))
    return out


def project_v_plan(p: PrismParams, X: torch.Tensor, Wv: torch.Tensor, a: torch.Tensor | None = None,
                   V: torch.Tensor | None = None, out: Plan | None = None, stream=None):
    """prism_project_v_plan: V = X Wv^T (bf16 [N, heads, head_dim]) with the
    plan computed from the zone statistics of the projection's own tiles.
    X bf16 [N, C], Wv bf16 [heads*head_dim, C].  Returns (V, plan)."""
    N = p.T * p.H * p.W
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise ValueError("X must be a 2-D tensor [N, C]")
    Cin = X.shape[1]
    _check_tensor(X, "X", torch.bfloat16, (N, Cin))
    _check_tensor(Wv, "Wv", torch.bfloat16, (p.heads * p.head_dim, Cin))
    if V is not None:
        _check_tensor(V, "V", torch.bfloat16, (N, p.heads, p.head_dim))
    if a is not None:
        _check_tensor(a, "a2v_norm", torch.float32, (N,))
    named = [("X", X), ("Wv", Wv), ("V", V), ("a2v_norm", a)] + (_check_plan(p, out) if out is not None else [])
    dev = _check_devices(named)
    made_v, made = V is None, out is None
    with torch.cuda.device(dev), _alloc_on(stream, dev):
        V = V if V is not None else torch.empty((N, p.heads, p.head_dim), dtype=torch.bfloat16, device=dev)
        out = out if out is not None else alloc_plan(p, dev)
        cs = out.c_struct()
        check(_lib.load().prism_project_v_plan(C.byref(p), _ptr(X), Cin, _ptr(Wv), _ptr(V), _ptr(a), C.byref(cs),
                                               _ptr(out.ws), out.ws.numel(), _stream(stream, dev)))
    _hand_over(stream, dev, V if made_v else None, *(out.tensors() if made else ()))
    return V, out


@dataclass
class Selection:
    """Output of prism_select (device tensors): a CSR over rows h*NB + i
    (head h, query block i) with row_ptr i32 [heads*NB + 1] and col i32
    [capacity] (selected key blocks, ascending; the first nnz entries are
    valid), and optionally its transpose col_ptr / row (needed by the
    backward); ws the call's workspace."""
    p: PrismParams
    row_ptr: torch.Tensor
    col: torch.Tensor
    col_ptr: torch.Tensor | None
    row: torch.Tensor | None
    nnz: int
    ws: torch.Tensor

    def tensors(self):
        return (self.row_ptr, self.col, self.col_ptr, self.row, self.ws)

    def c_struct(self) -> PrismSelect:
        return PrismSelect(self.row_ptr.data_ptr(), self.col.data_ptr(), self.col.numel(), self.nnz,
                           self.col_ptr.data_ptr() if self.col_ptr is not None else None,
                           self.row.data_ptr() if self.row is not None else None)


def alloc_select(p: PrismParams, device, cap: int, transpose: bool = True) -> Selection:
    _, _, NB = _sizes(p)
    lib = _lib.load()
    ws = _workspace(lib.prism_select_workspace_size(C.byref(p)), device)
    rows = p.heads * NB + 1
    return Selection(p, torch.empty((rows,), dtype=torch.int32, device=device),
                     torch.empty((max(cap, 1),), dtype=torch.int32, device=device),
                     torch.empty((rows,), dtype=torch.int32, device=device) if transpose else None,
                     torch.empty((max(cap, 1),), dtype=torch.int32, device=device) if transpose else None,
                     0, ws)


def _check_selection(p: PrismParams, sel: Selection, transpose: bool):
    """Structural checks of a selection against the call's grid; returns its
    named tensors for the device check."""
    if not isinstance(sel, Selection):
        raise TypeError(f"selection must be an api.Selection, got {type(sel).__name__}")
    _check_grid(p, sel.p, "the selection")
    _, _, NB = _sizes(p)
    rows = p.heads * NB + 1
    if not isinstance(sel.col, torch.Tensor) or sel.col.dim() != 1:
        raise ValueError("selection.col must be a 1-D tensor")
    cap = sel.col.numel()
    _check_tensor(sel.row_ptr, "selection.row_ptr", torch.int32, (rows,))
    _check_tensor(sel.col, "selection.col", torch.int32, (cap,))
    if (sel.col_ptr is None) != (sel.row is None):
        raise ValueError("selection.col_ptr and selection.row must both be set or both be None")
    if sel.col_ptr is not None:
        _check_tensor(sel.col_ptr, "selection.col_ptr", torch.int32, (rows,))
        _check_tensor(sel.row, "selection.row", torch.int32, (cap,))
    elif transpose:
        raise ValueError("the backward needs the selection's transpose (select(..., transpose=True))")
    if not 0 <= sel.nnz <= cap:
        raise ValueError(f"selection.nnz = {sel.nnz} exceeds its capacity {cap}")
    _check_workspace(sel.ws, "selection.ws")
    return [("selection.row_ptr", sel.row_ptr), ("selection.col", sel.col), ("selection.col_ptr", sel.col_ptr),
            ("selection.row", sel.row), ("selection.ws", sel.ws)]


def default_capacity(p: PrismParams) -> int:
    _, _, NB = _sizes(p)
    k = p.topk_abs if p.topk_abs > 0 else max(1, math.ceil(p.topk_frac * NB))
    return p.heads * NB * min(NB, 2 * k + 64)


def select(p: PrismParams, pl: Plan, Q: torch.Tensor, K: torch.Tensor, out: Selection | None = None,
           cap: int | None = None, transpose: bool = True, stream=None) -> Selection:
    """prism_select: block means, block scores, hybrid Top-k U Top-p (CSR and
    optionally its transpose).  Grows the output once if its capacity is short."""
    N = p.T * p.H * p.W
    _check_tensor(Q, "Q", torch.bfloat16, (N, p.heads, p.head_dim))
    _check_tensor(K, "K", torch.bfloat16, (N, p.heads, p.head_dim))
    named = [("Q", Q), ("K", K)] + _check_plan(p, pl)
    if out is not None:
        named += _check_selection(p, out, False)
    dev = _check_devices(named)
    lib = _lib.load()
    made, made_col = out is None, False
    with torch.cuda.device(dev), _alloc_on(stream, dev):
        if out is None:
            out = alloc_select(p, dev, cap if cap is not None else default_capacity(p), transpose)
        cpl = pl.c_struct()
        for attempt in range(2):
            cs = out.c_struct()
            rc = lib.prism_select(C.byref(p), C.byref(cpl), _ptr(Q), _ptr(K), C.byref(cs), _ptr(out.ws),
                                  out.ws.numel(), _stream(stream, dev))
            if rc == _lib.PRISM_ERR_CAPACITY and attempt == 0 and out.col.numel() < cs.nnz <= 0x7fffffff:
                need = int(cs.nnz)
                made_col = True
                out.col = torch.empty((need,), dtype=torch.int32, device=dev)
                if out.row is not None:
                    out.row = torch.empty((need,), dtype=torch.int32, device=dev)
                continue
            check(rc)
            break
    out.nnz = int(cs.nnz)
    _hand_over(stream, dev, *(out.tensors() if made else (out.col, out.row) if made_col else ()))
    return out


@dataclass
class FwdResult:
    """Output of prism_attn_fwd: O bf16 [N, heads, D] (natural order), lse
    f32 [heads, N] (natural log), ws the call's workspace (its status word
    says whether a kernel recorded an error), O_res the bf16 rounding
    residual of O, or None."""
    O: torch.Tensor
    lse: torch.Tensor
    ws: torch.Tensor
    O_res: torch.Tensor | None = None


def attn_fwd(p: PrismParams, pl: Plan, sel: Selection, Q, K, V, O=None, lse=None, ws=None, O_res=None,
             residual: bool = True, stream=None) -> FwdResult:
    """prism_attn_fwd: attention over the selected blocks; O natural order,
    lse [heads, N]; with `residual`, also O's bf16 rounding residual for the
    backward's Delta."""
    N = p.T * p.H * p.W
    shape = (N, p.heads, p.head_dim)
    for name, t in (("Q", Q), ("K", K), ("V", V)):
        _check_tensor(t, name, torch.bfloat16, shape)
    if O is not None:
        _check_tensor(O, "O", torch.bfloat16, shape)
    if residual and O_res is not None:
        _check_tensor(O_res, "O_res", torch.bfloat16, shape)
    if lse is not None:
        _check_tensor(lse, "lse", torch.float32, (p.heads, N))
    if ws is not None:
        _check_workspace(ws, "ws")
    named = [("Q", Q), ("K", K), ("V", V), ("O", O), ("O_res", O_res if residual else None), ("lse", lse),
             ("ws", ws)] + _check_plan(p, pl) + _check_selection(p, sel, False)
    dev = _check_devices(named)
    lib = _lib.load()
    given = (O, O_res, lse, ws)
    with torch.cuda.device(dev), _alloc_on(stream, dev):
        O = O if O is not None else torch.empty_like(Q)
        if residual and O_res is None:
            O_res = torch.empty_like(Q)
        lse = lse if lse is not None else torch.empty((p.heads, N), dtype=torch.float32, device=dev)
        ws = ws if ws is not None else _workspace(lib.prism_attn_workspace_size(C.byref(p), 0), dev)
        cpl, cs = pl.c_struct(), sel.c_struct()
        check(lib.prism_attn_fwd(C.byref(p), C.byref(cpl), C.byref(cs), _ptr(Q), _ptr(K), _ptr(V), _ptr(O),
                                 _ptr(O_res) if residual else None, _ptr(lse), _ptr(ws), ws.numel(),
                                 _stream(stream, dev)))
    _hand_over(stream, dev, *(t for g, t in zip(given, (O, O_res, lse, ws)) if g is None))
    return FwdResult(O, lse, ws, O_res if residual else None)


def attn_bwd(p: PrismParams, pl: Plan, sel: Selection, Q, K, V, O, dO, lse, grad_fp32=False, out=None, ws=None,
             O_res=None, stream=None, deterministic=False):
    """prism_attn_bwd: dQ, dK, dV through the selected blocks (natural order).
    Pass the forward's O_res for an fp32-accurate Delta.  deterministic=False
    (head_dim 128) takes the fused kernel, whose dQ is summed by fp32
    reductions in no fixed order; True takes the two-kernel path, bitwise
    reproducible."""
    N = p.T * p.H * p.W
    shape = (N, p.heads, p.head_dim)
    for name, t in (("Q", Q), ("K", K), ("V", V), ("O", O), ("dO", dO)):
        _check_tensor(t, name, torch.bfloat16, shape)
    if O_res is not None:
        _check_tensor(O_res, "O_res", torch.bfloat16, shape)
    _check_tensor(lse, "lse", torch.float32, (p.heads, N))
    dt = torch.float32 if grad_fp32 else torch.bfloat16
    if out is not None:
        if len(out) != 3:
            raise ValueError("out must hold the three gradients (dQ, dK, dV)")
        for name, t in zip(("dQ", "dK", "dV"), out):
            _check_tensor(t, name, dt, shape)
    if ws is not None:
        _check_workspace(ws, "ws")
    named = [("Q", Q), ("K", K), ("V", V), ("O", O), ("dO", dO), ("O_res", O_res), ("lse", lse), ("ws", ws)]
    if out is not None:
        named += list(zip(("dQ", "dK", "dV"), out))
    named += _check_plan(p, pl) + _check_selection(p, sel, True)
    dev = _check_devices(named)
    lib = _lib.load()
    made = out is None
    with torch.cuda.device(dev), _alloc_on(stream, dev):
        if out is None:
            out = tuple(torch.empty(shape, dtype=dt, device=dev) for _ in range(3))
        ws = ws if ws is not None else _workspace(lib.prism_attn_workspace_size(C.byref(p), 1), dev)
        cpl, cs = pl.c_struct(), sel.c_struct()
        dQ, dK, dV = out
        check(lib.prism_attn_bwd(C.byref(p), C.byref(cpl), C.byref(cs), _ptr(Q), _ptr(K), _ptr(V), _ptr(O),
                                 _ptr(O_res), _ptr(dO), _ptr(lse), _ptr(dQ), _ptr(dK), _ptr(dV),
                                 int(bool(grad_fp32)), int(bool(deterministic)), _ptr(ws), ws.numel(),
                                 _stream(stream, dev)))
    _hand_over(stream, dev, *(out if made else ()))
    return dQ, dK, dV


def workspace_status(ws: torch.Tensor, stream=None) -> int:
    """The status word a call left in its workspace (PRISM_OK, or the error a
    kernel recorded, e.g. PRISM_ERR_TIMEOUT or PRISM_ERR_RANGE)."""
    _check_workspace(ws, "ws")
    dev = _check_devices([("ws", ws)])
    with torch.cuda.device(dev):
        return _lib.load().prism_workspace_status(_ptr(ws), _stream(stream, dev))


# ----------------------------------------------------------------------------- linear maps and checkpoints
# These calls can be a few microseconds of GPU work, so what surrounds them is
# kept short: no device switch where the tensors' device is current already, the
# current stream by its raw handle, addresses as plain integers, sizes of new
# tensors as separate arguments (0.7 us less than a tuple).
def _on(dev, stream):
    if stream is not None:
        there = _alloc_on(stream, dev)  # may refuse the stream: before anything is entered
        both = contextlib.ExitStack()
        both.enter_context(torch.cuda.device(dev))
        both.enter_context(there)
        return both
    return _HERE if dev.index == torch._C._cuda_getDevice() else torch.cuda.device(dev)


def _handle(stream, dev) -> int:
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev.index)


def _addr(t):
    return None if t is None else t.data_ptr()


# ----------------------------------------------------------------------------- 8-bit activation checkpoints
@dataclass
class Ckpt8:
    """An activation [n, width] held in 8 bits (prism_ckpt8_t): codes i8
    [n, ld] and scales u8 [n, ld / 32], ld = width rounded up to a multiple of
    128; a value is code * 2^(scale - 127)."""
    codes: torch.Tensor
    scales: torch.Tensor
    width: int

    def c_struct(self) -> PrismCkpt8:
        return PrismCkpt8(self.codes.data_ptr(), self.scales.data_ptr(), self.codes.shape[1])


def alloc_ckpt8(n: int, width: int, device) -> Ckpt8:
    ld = (width + 127) // 128 * 128
    return Ckpt8(torch.empty(n, ld, dtype=torch.int8, device=device),
                 torch.empty(n, ld // 32, dtype=torch.uint8, device=device), width)


def _check_ckpt8(c, name, n, width):
    if not isinstance(c, Ckpt8):
        raise TypeError(f"{name} must be an api.Ckpt8, got {type(c).__name__}")
    if c.width != width:
        raise ValueError(f"{name} holds {c.width} channels, the call needs {width}")
    if width > 0x7fffffff:
        raise ValueError(f"{name} has {width} channels; the library holds them in 32 bits")
    ld = (width + 127) // 128 * 128
    _check_tensor(c.codes, name + ".codes", torch.int8, (n, ld))
    _check_tensor(c.scales, name + ".scales", torch.uint8, (n, ld // 32))
    return [(name + ".codes", c.codes), (name + ".scales", c.scales)]


def _check_rows(t, name, shape=None):
    """A 2-D bf16 tensor whose rows may be strided (contiguous within a row);
    returns its row stride in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    got = t.shape
    if len(got) != 2 or (shape is not None and got != shape):
        want = "two dimensions" if shape is None else f"shape {tuple(shape)}"
        raise ValueError(f"{name} must have {want}, got {tuple(got)}")
    rows, cols = got
    if cols > 0x7fffffff:
        raise ValueError(f"{name} has {cols} channels; the library holds them in 32 bits")
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} rows must be contiguous")
    if rows <= 1:
        return cols
    if ld < cols:
        raise ValueError(f"{name} rows overlap (stride {ld}, {cols} channels)")
    return ld


def ckpt8_pack(x: torch.Tensor, out: Ckpt8 | None = None, stream=None) -> Ckpt8:
    """prism_ckpt8_pack: the 8-bit checkpoint of a bf16 activation x [n, width]
    (rows may be strided; width a multiple of 8)."""
    ld = _check_rows(x, "x")
    n, width = x.shape
    named = [("x", x)] + (_check_ckpt8(out, "out", n, width) if out is not None else [])
    dev = _check_devices(named)
    made = out is None
    with _on(dev, stream):
        out = out if out is not None else alloc_ckpt8(n, width, dev)
        cs = out.c_struct()
        check(_lib.load().prism_ckpt8_pack(_addr(x), n, width, ld, C.byref(cs), _handle(stream, dev)))
    if stream is not None and made:
        _hand_over(stream, dev, out.codes, out.scales)
    return out


def ckpt8_unpack(c: Ckpt8, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """prism_ckpt8_unpack: the activation a checkpoint holds, bf16 [n, width]
    (into `out`, whose rows may be strided)."""
    if not isinstance(c, Ckpt8) or not isinstance(c.codes, torch.Tensor) or c.codes.dim() != 2:
        raise TypeError("c must be an api.Ckpt8")
    n = c.codes.shape[0]
    named = _check_ckpt8(c, "c", n, c.width)
    ld = c.width
    if out is not None:
        ld = _check_rows(out, "out", (n, c.width))
        named.append(("out", out))
    dev = _check_devices(named)
    made = out is None
    with _on(dev, stream):
        out = out if out is not None else torch.empty(n, c.width, dtype=torch.bfloat16, device=dev)
        cs = c.c_struct()
        check(_lib.load().prism_ckpt8_unpack(C.byref(cs), n, c.width, _addr(out), ld, _handle(stream, dev)))
    if stream is not None and made:
        _hand_over(stream, dev, out)
    return out


# ----------------------------------------------------------------------------- linear maps
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = 0, 1, 2, 3  # activations of the linear map (gelu: tanh form)


@dataclass
class LinearResult:
    """Output of prism_linear_fwd: Y bf16 [n, out]; Z the saved
    pre-activation (bf16 tensor, Ckpt8 or None); ws the call's workspace
    (its status word says whether a kernel gave up on a wait)."""
    Y: torch.Tensor
    Z: torch.Tensor | Ckpt8 | None
    ws: torch.Tensor


@dataclass
class LinearGrads:
    """Output of prism_linear_bwd: dX bf16 [n, in], dW [out, in], db [out]
    (bf16 or fp32; None where not asked for), ws the call's workspace, or a copy
    of its header with the status word where the call allocated more than
    _KEPT_WORKSPACE bytes: dZ, partial sums and a restored X are of no further
    use."""
    dX: torch.Tensor | None
    dW: torch.Tensor | None
    db: torch.Tensor | None
    ws: torch.Tensor


# A backward's workspace holds dZ and perhaps X, as large as the activations.  Above this
# size it is given back with the call; the copy of its header takes 2 to 4 us, beside calls
# of 100 us or more.
_KEPT_WORKSPACE = 1 << 26


def _describe(n, cin, cout, act) -> PrismLinear:
    """The call's description.  What it holds in 32 bits is checked here: ctypes
    would drop the upper ones, and the library see another size or activation."""
    if not (-1 << 31 <= cin < 1 << 31 and -1 << 31 <= cout < 1 << 31):
        raise ValueError(f"in and out are at most 65536 channels, got {cin}, {cout}")
    if not ACT_NONE <= act <= ACT_GELU:
        raise ValueError(f"act must be one of ACT_NONE .. ACT_GELU (0..3), got {act}")
    if not -1 << 63 <= n < 1 << 63:
        raise ValueError(f"n must be below 2^30 tokens, got {n}")
    return PrismLinear(n, cin, cout, act)


def linear_workspace_size(n: int, cin: int, cout: int, act: int = ACT_NONE, backward: bool = False,
                          x8: bool = False) -> int:
    """Bytes of the `ws` buffer linear_fwd / linear_bwd takes for n tokens (x8:
    linear_bwd with X as a Ckpt8)."""
    mode = (2 if x8 else 1) if backward else 0
    size = _lib.load().prism_linear_workspace_size(C.byref(_describe(n, cin, cout, act)), mode)
    if size == 0:
        raise _lib.PrismError(_lib.PRISM_ERR_INVALID_ARG, _lib.load().prism_last_error().decode(errors="replace"))
    return size


def linear_fwd(X: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None, act: int = ACT_NONE,
               residual: torch.Tensor | None = None, save: str | None = None, Y: torch.Tensor | None = None,
               Z: torch.Tensor | Ckpt8 | None = None, ws: torch.Tensor | None = None, stream=None) -> LinearResult:
    """prism_linear_fwd: Y = act(X W^T + bias) + residual.  X bf16 [n, in], W
    bf16 [out, in], bias bf16 [out], residual bf16 [n, out]; X, residual and Y
    rows may be strided.  save = "bf16" or "ckpt8" keeps the pre-activation for
    linear_bwd (into Z when given).  Y may be the residual itself; otherwise the
    library refuses outputs that share memory with an input or one another."""
    ldx = _check_rows(X, "X")
    n, cin = X.shape
    if not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise ValueError("W must be a 2-D tensor [out, in]")
    cout = W.shape[0]
    _check_tensor(W, "W", torch.bfloat16, (cout, cin))
    named = [("X", X), ("W", W), ("bias", bias), ("residual", residual), ("Y", Y), ("ws", ws)]
    if bias is not None:
        _check_tensor(bias, "bias", torch.bfloat16, (cout,))
    ldr = _check_rows(residual, "residual", (n, cout)) if residual is not None else 0
    ldy = cout
    if Y is not None:
        ldy = _check_rows(Y, "Y", (n, cout))
        if n > 0 and Y.data_ptr() == X.data_ptr():
            raise ValueError("Y may not be X (every output channel reads all of X's)")
    if save not in (None, "bf16", "ckpt8"):
        raise ValueError(f'save must be None, "bf16" or "ckpt8", got {save!r}')
    if Z is not None:
        if save is None:
            raise ValueError("Z is given but save is None")
        if save == "bf16":
            _check_tensor(Z, "Z", torch.bfloat16, (n, cout))
            named.append(("Z", Z))
        else:
            named += _check_ckpt8(Z, "Z", n, cout)
    if ws is not None:
        _check_workspace(ws, "ws")
    l = _describe(n, cin, cout, act)
    dev = _check_devices(named)
    lib = _lib.load()
    given = (Y, Z, ws)
    with _on(dev, stream):
        Y = Y if Y is not None else torch.empty(n, cout, dtype=torch.bfloat16, device=dev)
        if Z is None and save is not None:
            Z = torch.empty_like(Y, memory_format=torch.contiguous_format) if save == "bf16" else \
                alloc_ckpt8(n, cout, dev)
        ws = ws if ws is not None else torch.empty(256, dtype=torch.uint8, device=dev)
        z8 = Z.c_struct() if save == "ckpt8" else None
        check(lib.prism_linear_fwd(C.byref(l), X.data_ptr(), ldx, W.data_ptr(), _addr(bias), _addr(residual), ldr,
                                   Y.data_ptr(), ldy,
                                   _addr(Z) if save == "bf16" else None, C.byref(z8) if z8 is not None else None,
                                   ws.data_ptr(), ws.numel(), _handle(stream, dev)))
    if stream is not None:
        z = (Z.codes, Z.scales) if save == "ckpt8" else (Z,)
        _hand_over(stream, dev, *((Y,) if given[0] is None else ()), *(z if given[1] is None else ()),
                   *((ws,) if given[2] is None else ()))
    return LinearResult(Y, Z, ws)


def linear_bwd(dY: torch.Tensor, X: torch.Tensor | Ckpt8 | None, W: torch.Tensor | None,
               Z: torch.Tensor | Ckpt8 | None = None, act: int = ACT_NONE, need=("dX", "dW", "db"),
               grad_fp32: bool = False, out=None, ws: torch.Tensor | None = None, stream=None) -> LinearGrads:
    """prism_linear_bwd: the gradients named in `need` of linear_fwd, from dY
    bf16 [n, out], the forward's X [n, in] (bf16 or a Ckpt8; needed for dW), W
    (needed for dX) and, with an activation, the saved pre-activation Z (bf16 or
    a Ckpt8).  dX is bf16; dW and db bf16, or fp32 with grad_fp32 (with silu
    or gelu, dW's operand dY * act'(Z) is rounded to bf16, and the fp32 dW is as
    accurate as that: about 1.7e-3 of its norm; otherwise 5e-7).  `out` may
    hold (dX, dW, db) buffers, None entries allocated; the library refuses
    buffers that share memory with what the call reads (X's for dX unless `need`
    leaves dW out) or with one another.  The residual's gradient is dY itself."""
    lddy = _check_rows(dY, "dY")
    n, cout = dY.shape
    want_x, want_w, want_b = "dX" in need, "dW" in need, "db" in need
    if isinstance(need, str) or len(need) == 0 or len(need) != want_x + want_w + want_b:
        raise ValueError(f'need must name some of "dX", "dW", "db", once each, got {need!r}')
    if want_x and W is None:
        raise ValueError("dX needs W")
    if want_w and X is None:
        raise ValueError("dW needs X")
    x8 = isinstance(X, Ckpt8)
    if W is not None:
        if not isinstance(W, torch.Tensor) or W.dim() != 2:
            raise ValueError("W must be a 2-D tensor [out, in]")
        cin = W.shape[1]
        _check_tensor(W, "W", torch.bfloat16, (cout, cin))
    elif x8:
        cin = X.width
    elif X is not None:
        _check_rows(X, "X")
        cin = X.shape[1]
    else:
        cin = 8  # only db: the input's width does not matter
    named = [("dY", dY), ("W", W)]
    ldx = ldz = 0
    if x8:
        named += _check_ckpt8(X, "X", n, cin)
    elif X is not None:
        ldx = _check_rows(X, "X", (n, cin))
        named.append(("X", X))
    z8 = False
    if act == ACT_NONE:
        Z = None
    elif Z is None:
        raise ValueError("the activation's gradient needs Z")
    elif isinstance(Z, Ckpt8):
        z8 = True
        named += _check_ckpt8(Z, "Z", n, cout)
    else:
        ldz = _check_rows(Z, "Z", (n, cout))
        named.append(("Z", Z))
    dt = torch.float32 if grad_fp32 else torch.bfloat16
    dX = dW = db = None
    if out is not None:
        if len(out) != 3:
            raise ValueError("out must hold three entries (dX, dW, db)")
        dX, dW, db = out
        for name, t, wanted, dtype, shape in (("dX", dX, want_x, torch.bfloat16, (n, cin)),
                                              ("dW", dW, want_w, dt, (cout, cin)), ("db", db, want_b, dt, (cout,))):
            if t is not None:
                if not wanted:
                    raise ValueError(f"out holds {name}, which need does not name")
                _check_tensor(t, name, dtype, shape)
                named.append((name, t))
        if dX is not None and n > 0 and dX.data_ptr() == dY.data_ptr():
            raise ValueError("dX may not be dY (every input channel reads all of dY's)")
    if ws is not None:
        _check_workspace(ws, "ws")
        named.append(("ws", ws))
    l = _describe(n, cin, cout, act)
    dev = _check_devices(named)
    lib = _lib.load()
    given = (dX, dW, db, ws)
    with _on(dev, stream):
        if want_x and dX is None:
            dX = torch.empty(n, cin, dtype=torch.bfloat16, device=dev)
        if want_w and dW is None:
            dW = torch.empty(cout, cin, dtype=dt, device=dev)
        if want_b and db is None:
            db = torch.empty(cout, dtype=dt, device=dev)
        if ws is None:
            ws = _workspace(lib.prism_linear_workspace_size(C.byref(l), 2 if x8 else 1), dev)
        cx = C.byref(X.c_struct()) if x8 else None
        cz = C.byref(Z.c_struct()) if z8 else None
        check(lib.prism_linear_bwd(C.byref(l), dY.data_ptr(), lddy, None if x8 else _addr(X), ldx, cx, _addr(W),
                                   None if z8 else _addr(Z), ldz, cz, _addr(dX), _addr(dW), _addr(db),
                                   1 if grad_fp32 else 0, ws.data_ptr(), ws.numel(), _handle(stream, dev)))
        if given[3] is None and ws.numel() > _KEPT_WORKSPACE and (stream is None or isinstance(stream, torch.cuda.Stream)):
            ws = ws[:256].clone()
    if stream is not None:
        _hand_over(stream, dev, *(t for g, t in zip(given, (dX, dW, db, ws)) if g is None))
    return LinearGrads(dX, dW, db, ws)
