"""Sparse Mixture-of-Experts layer forward for NVIDIA B200 (sm_100a).

Thin ctypes binding of ``libmoe_b200.so`` (declared in ``include/moe_b200.h``).
Functions take CUDA torch tensors and marshal their device pointers, sizes and
the current CUDA stream into the C ABI; every step of the layer runs in the
library's CUDA kernels.  PyTorch only provides device memory and streams.

There is no CPU path: importing this package fails loudly if the library is
missing, and every call requires CUDA tensors.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# MOE_B200_CHECK_BOUNDS=1: load the bounds-checked build (moe_bounds_checked)
CHECK_BOUNDS = os.environ.get("MOE_B200_CHECK_BOUNDS", "0") == "1"
LIB_PATH = os.path.join(_PKG, "libmoe_b200_checked.so" if CHECK_BOUNDS else "libmoe_b200.so")

MOE_OK = 0
ERRORS = {-1: "MOE_ERR_INVALID_ARGUMENT", -2: "MOE_ERR_UNSUPPORTED", -3: "MOE_ERR_ALIGNMENT",
          -4: "MOE_ERR_WORKSPACE", -5: "MOE_ERR_CUDA"}
DTYPE_BF16, DTYPE_F32 = 0, 1
ROUTE_TOPK, ROUTE_RRE = 0, 1
STATUS_TIMEOUT, STATUS_BAD_DOMAIN, STATUS_BAD_COUNTS, STATUS_BAD_INDEX = 1, 2, 4, 8
STATUS_BAD_LOGIT, STATUS_NONFINITE = 16, 32
FFN_WORKSPACE_ZEROED = 1

# every entry point the header declares, with its ctypes signature
_i32, _i64, _u64, _sz, _vp, _dbl = (ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64,
                                    ctypes.c_size_t, ctypes.c_void_p, ctypes.c_double)


class MoEConfig(ctypes.Structure):
    """Mirror of ``moe_config`` (56 bytes)."""
    _fields_ = [("T", _i64), ("d_model", _i32), ("d_ff", _i32), ("E", _i32), ("k", _i32),
                ("capacity", _i32), ("mode", _i32), ("num_groups", _i32), ("dtype", _i32),
                ("expert", _i32), ("reserved", _i32), ("seed", _u64)]


class WorkspaceMap(ctypes.Structure):
    """Mirror of ``moe_workspace_map``."""
    _fields_ = [(n, _sz) for n in ("logits", "expert_idx", "gate", "slot", "kept", "tok_of_row",
                                   "arrivals", "kept_cnt", "n_dropped", "scratch", "ffn_sync", "xe",
                                   "H", "ye",
                                   "total")]


class RouteConfig(ctypes.Structure):
    """Mirror of ``moe_route_config`` (48 bytes)."""
    _fields_ = [("T", _i64), ("E", _i32), ("k", _i32), ("score", _i32), ("num_groups", _i32),
                ("top_groups", _i32), ("group_top", _i32), ("renorm", _i32), ("dtype", _i32),
                ("scale", _dbl)]


class AdamWConfig(ctypes.Structure):
    """Mirror of ``moe_adamw_config`` (64 bytes)."""
    _fields_ = [("lr", _dbl), ("beta1", _dbl), ("beta2", _dbl), ("eps", _dbl),
                ("weight_decay", _dbl), ("max_norm", _dbl), ("step", _i64), ("grad_dtype", _i32),
                ("state_bits", _i32)]


_PCFG = ctypes.POINTER(MoEConfig)
_PRCFG, _PACFG = ctypes.POINTER(RouteConfig), ctypes.POINTER(AdamWConfig)
_PVP = ctypes.POINTER(ctypes.c_void_p)
SIGNATURES = {
    "moe_abi_version": ([], _i32),
    "moe_config_size": ([], _sz),
    "moe_workspace_map_size": ([], _sz),
    "moe_error_string": ([_i32], ctypes.c_char_p),
    "moe_last_error": ([], ctypes.c_char_p),
    "moe_capacity": ([_i64, _i32, _dbl], _i32),
    "moe_config_check": ([_PCFG], _i32),
    "moe_assign_workspace_size": ([_PCFG], _sz),
    "moe_workspace_layout": ([_PCFG, ctypes.POINTER(WorkspaceMap)], _i32),
    "moe_workspace_size": ([_PCFG], _sz),
    "sparseclip_workspace_size": ([_i32, _i32], _sz),
    "moe_router": ([_PCFG, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_topk_assign": ([_PCFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp,
                         _vp], _i32),
    "moe_dispatch": ([_PCFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_ffn_workspace_size": ([_PCFG], _sz),
    "moe_expert_ffn": ([_PCFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp], _i32),
    "moe_expert_ffn_ex": ([_PCFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, ctypes.c_uint32, _vp,
                           _vp], _i32),
    "moe_set_wait_limit_ns": ([_u64], None),
    "moe_wait_limit_ns": ([], _u64),
    "moe_combine": ([_PCFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_bounds_checked": ([], _i32),
    "moe_layer_forward": ([_PCFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp, _vp],
                          _i32),
    "moe_aux_workspace_size": ([_PCFG], _sz),
    "moe_aux_loss": ([_PCFG, _vp, _dbl, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "sparseclip_norm": ([_vp, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _vp, _sz, _vp], _i32),
    "sparseclip_norm_noalloc": ([_vp, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _vp], _i32),
    "sparseclip_clip": ([_vp, _vp, _i32, _vp, _vp, _i32, _i32, _dbl, _vp, _vp, _sz, _vp], _i32),
    "moe_route_config_size": ([], _sz),
    "moe_adamw_config_size": ([], _sz),
    "moe_route": ([_PRCFG, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_route_backward": ([_PRCFG, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_assign": ([_PCFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_dispatch_backward": ([_PCFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_combine_backward": ([_PCFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_adamw_check": ([_PACFG, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_adamw_step": ([_PACFG, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
                       _i32),
    "moe_ep_ffn_config": ([_PCFG, _i32, _PCFG], _i32),
    "moe_ep_dispatch": ([_PCFG, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _PVP, _vp, _vp, _vp], _i32),
    "moe_ep_combine": ([_PCFG, _i32, _i32, _PVP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
}


def _load_library():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python sparse_mixture_experts_fwd_b200/build.py` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    assert lib.moe_config_size() == ctypes.sizeof(MoEConfig), "moe_config layout mismatch"
    assert lib.moe_workspace_map_size() == ctypes.sizeof(WorkspaceMap), "workspace map mismatch"
    assert lib.moe_route_config_size() == ctypes.sizeof(RouteConfig), "moe_route_config mismatch"
    assert lib.moe_adamw_config_size() == ctypes.sizeof(AdamWConfig), "moe_adamw_config mismatch"
    return lib


lib = _load_library()


class MoEError(RuntimeError):
    def __init__(self, code: int, where: str):
        detail = lib.moe_last_error().decode()
        super().__init__(f"{where}: {ERRORS.get(code, code)} ({detail})")
        self.code = code


def _check(code: int, where: str):
    if code != MOE_OK:
        raise MoEError(code, where)


def _dtype_code(dtype) -> int:
    if dtype == torch.bfloat16:
        return DTYPE_BF16
    if dtype == torch.float32:
        return DTYPE_F32
    raise TypeError(f"unsupported activation dtype {dtype}")


def _ptr(t, name):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# torch's own handles where they are there (a torch built without CUDA has none: then the first
# call raises torch's error, as its public functions do)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    # the handle alone: building torch's Stream object costs 3 us a call
    return _current_stream(_current_device())


def capacity(T: int, E: int, capacity_factor: float) -> int:
    """Eq. (3): floor(T / E * capacity_factor)."""
    return int(lib.moe_capacity(T, E, capacity_factor))


EXPERTS = {"relu": 0, "geglu": 1}


def make_config(T, d_model, d_ff, E, k, capacity_, *, dtype=torch.bfloat16, mode="topk",
                num_groups=1, seed=0, expert="relu") -> MoEConfig:
    """expert: "relu" (W1 [E, f, d]) or "geglu" (W1 [E, 2f, d], bf16 only)."""
    return MoEConfig(T=T, d_model=d_model, d_ff=d_ff, E=E, k=k, capacity=capacity_,
                     mode=ROUTE_TOPK if mode == "topk" else ROUTE_RRE, num_groups=num_groups,
                     dtype=_dtype_code(dtype), expert=EXPERTS[expert], reserved=0, seed=seed)


def config_check(cfg: MoEConfig):
    _check(lib.moe_config_check(ctypes.byref(cfg)), "moe_config_check")


def workspace_layout(cfg: MoEConfig) -> WorkspaceMap:
    m = WorkspaceMap()
    _check(lib.moe_workspace_layout(ctypes.byref(cfg), ctypes.byref(m)), "moe_workspace_layout")
    return m


def workspace_size(cfg: MoEConfig) -> int:
    return int(workspace_layout(cfg).total)


def assign_workspace_size(cfg: MoEConfig) -> int:
    config_check(cfg)
    return int(lib.moe_assign_workspace_size(ctypes.byref(cfg)))


def _act_dtype(cfg):
    return torch.bfloat16 if cfg.dtype == DTYPE_BF16 else torch.float32


def router(cfg, x, Wr, bias=None, logits=None, status=None, stream=None):
    if logits is None:
        logits = torch.empty(cfg.T, cfg.E, dtype=torch.float32, device=x.device)
    _check(lib.moe_router(ctypes.byref(cfg), _ptr(x, "x"), _ptr(Wr, "Wr"), _ptr(bias, "bias"),
                          _ptr(logits, "logits"), _ptr(status, "status"), _stream(stream)),
           "moe_router")
    return logits


def aux_workspace_size(cfg: MoEConfig) -> int:
    return int(lib.moe_aux_workspace_size(ctypes.byref(cfg)))


def aux_loss(cfg, logits, alpha=1e-2, workspace=None, stream=None):
    """Switch load-balancing loss and routing entropy from fp32 logits [T, E].

    Returns device float64 tensors: out [2] (loss, entropy), f [E], P [E]."""
    dev = logits.device
    out = torch.empty(2, dtype=torch.float64, device=dev)
    f = torch.empty(cfg.E, dtype=torch.float64, device=dev)
    P = torch.empty(cfg.E, dtype=torch.float64, device=dev)
    if workspace is None:
        workspace = torch.empty(max(256, aux_workspace_size(cfg)), dtype=torch.uint8, device=dev)
    _check(lib.moe_aux_loss(ctypes.byref(cfg), _ptr(logits, "logits"), float(alpha),
                            _ptr(out, "out"), _ptr(f, "f"), _ptr(P, "P"), _ptr(workspace, "workspace"),
                            workspace.numel(), _stream(stream)), "moe_aux_loss")
    return out, f, P


def topk_assign(cfg, logits=None, domain_id=None, out=None, workspace=None, status=None,
                stream=None):
    """Returns a dict: expert_idx, gate, slot, kept, tok_of_row, arrivals, kept_cnt, n_dropped."""
    dev = (logits if logits is not None else domain_id).device
    T, k, E, C = cfg.T, cfg.k, cfg.E, cfg.capacity
    o = out or {}
    o.setdefault("expert_idx", torch.empty(T, k, dtype=torch.int32, device=dev))
    o.setdefault("gate", torch.empty(T, k, dtype=torch.float32, device=dev))
    o.setdefault("slot", torch.empty(T, k, dtype=torch.int32, device=dev))
    o.setdefault("kept", torch.empty(T, k, dtype=torch.uint8, device=dev))
    o.setdefault("tok_of_row", torch.empty(max(1, E * C), dtype=torch.int32, device=dev))
    o.setdefault("arrivals", torch.empty(E, dtype=torch.int32, device=dev))
    o.setdefault("kept_cnt", torch.empty(E, dtype=torch.int32, device=dev))
    o.setdefault("n_dropped", torch.empty(1, dtype=torch.int32, device=dev))
    if workspace is None:
        workspace = torch.empty(max(256, assign_workspace_size(cfg)), dtype=torch.uint8, device=dev)
    _check(lib.moe_topk_assign(
        ctypes.byref(cfg), _ptr(logits, "logits"), _ptr(domain_id, "domain_id"),
        _ptr(o["expert_idx"], "expert_idx"), _ptr(o["gate"], "gate"), _ptr(o["slot"], "slot"),
        _ptr(o["kept"], "kept"), _ptr(o["tok_of_row"], "tok_of_row"),
        _ptr(o["arrivals"], "arrivals"), _ptr(o["kept_cnt"], "kept_cnt"),
        _ptr(o["n_dropped"], "n_dropped"), _ptr(workspace, "workspace"), workspace.numel(),
        _ptr(status, "status"), _stream(stream)), "moe_topk_assign")
    return o


def _choice_args(cfg, expert_idx, slot, kept):
    """Pointers of the per-choice arrays [T, k]."""
    shape = (cfg.T, cfg.k)
    return (_arg(expert_idx, "expert_idx", torch.int32, shape),
            _arg(slot, "slot", torch.int32, shape), _arg(kept, "kept", torch.uint8, shape))


def dispatch(cfg, x, expert_idx, slot, kept, xe=None, status=None, stream=None):
    if cfg.k > 2:  # the arrays' types and shapes are settled, as in ``assign``
        act, rows = _act_dtype(cfg), (cfg.E, cfg.capacity, cfg.d_model)
        if xe is None:
            xe = _empty(rows, act, x.device, stream)
        _check(lib.moe_dispatch(ctypes.byref(cfg), _arg(x, "x", act, (cfg.T, cfg.d_model)),
                                *_choice_args(cfg, expert_idx, slot, kept),
                                _arg_rows(xe, "xe", act, rows), _status(status),
                                _stream(stream)), "moe_dispatch")
        return xe
    if xe is None:
        xe = torch.empty(cfg.E, cfg.capacity, cfg.d_model, dtype=x.dtype, device=x.device)
    _check(lib.moe_dispatch(ctypes.byref(cfg), _ptr(x, "x"), _ptr(expert_idx, "expert_idx"),
                            _ptr(slot, "slot"), _ptr(kept, "kept"), _ptr(xe, "xe"),
                            _ptr(status, "status"), _stream(stream)), "moe_dispatch")
    return xe


def _arg(t, name, dtype, shape):
    """Device pointer of an argument whose dtype, shape and device are settled."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        dev = t.get_device()  # -1: a CPU tensor
        if dev >= 0 and dev == _current_device():
            return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    _ptr(t, name)
    raise ValueError(f"{name} is on {t.device}, the current device is "
                     f"cuda:{torch.cuda.current_device()}")


def _empty(shape, dtype, device, stream):
    """A new output, owned by the stream the call runs on."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=device)


def _arg_rows(t, name, dtype, rows):
    """An [E, C, d] buffer, or the same rows as [E * C, d]."""
    flat = (rows[0] * rows[1], rows[2])
    return _arg(t, name, dtype, flat if t.dim() == 2 else rows)


def _status(status):
    return None if status is None else _arg(status, "status", torch.int32, (1,))


SCORES = {"softmax": 0, "sigmoid": 1}


def make_route_config(T, E, k, *, score="softmax", num_groups=1, top_groups=None, group_top=1,
                      renorm=False, scale=1.0, dtype=torch.float32) -> RouteConfig:
    """How ``route`` scores and chooses (``moe_route_config``).  ``top_groups``: groups a token
    may choose from (all of them by default); ``dtype``: the logits'."""
    return RouteConfig(T=T, E=E, k=k, score=SCORES[score], num_groups=num_groups,
                       top_groups=num_groups if top_groups is None else top_groups,
                       group_top=group_top, renorm=int(renorm), dtype=_dtype_code(dtype),
                       scale=scale)


def route(rcfg, logits, bias=None, expert_idx=None, gate=None, status=None, stream=None):
    """Choices and weights from router logits [T, E]: (expert_idx [T, k] int32, gate [T, k] fp32).

    ``bias`` [E] fp32 enters the choice only.  Ties go to the lower group and expert; with a
    bias or group values of two experts, scores that fp64 cannot tell apart are ties.  A token
    with fewer than k experts left (the others masked by -inf) gets -1 and weight 0 for the
    rest."""
    T, E, k = rcfg.T, rcfg.E, rcfg.k
    lp = _arg(logits, "logits", _act_dtype(rcfg), (T, E))
    bp = None if bias is None else _arg(bias, "bias", torch.float32, (E,))
    if expert_idx is None:
        expert_idx = _empty((T, k), torch.int32, logits.device, stream)
    if gate is None:
        gate = _empty((T, k), torch.float32, logits.device, stream)
    _check(lib.moe_route(ctypes.byref(rcfg), lp, bp,
                         _arg(expert_idx, "expert_idx", torch.int32, (T, k)),
                         _arg(gate, "gate", torch.float32, (T, k)), _status(status),
                         _stream(stream)), "moe_route")
    return expert_idx, gate


def route_backward(rcfg, logits, expert_idx, dgate, dlogits=None, status=None, stream=None):
    """Gradient of ``route``'s weights with respect to the logits, the choices held fixed."""
    T, E, k = rcfg.T, rcfg.E, rcfg.k
    lp = _arg(logits, "logits", _act_dtype(rcfg), (T, E))
    if dlogits is None:
        dlogits = _empty((T, E), logits.dtype, logits.device, stream)
    _check(lib.moe_route_backward(ctypes.byref(rcfg), lp,
                                  _arg(expert_idx, "expert_idx", torch.int32, (T, k)),
                                  _arg(dgate, "dgate", torch.float32, (T, k)),
                                  _arg(dlogits, "dlogits", logits.dtype, (T, E)),
                                  _status(status), _stream(stream)), "moe_route_backward")
    return dlogits


def assign(cfg, expert_idx, out=None, status=None, stream=None):
    """Slots for given choices [T, k], k up to 16.  Returns a dict: slot, kept, tok_of_row
    [E * C], arrivals, kept_cnt, n_dropped (``out`` may supply any of them)."""
    T, k, E, C = cfg.T, cfg.k, cfg.E, cfg.capacity
    ep = _arg(expert_idx, "expert_idx", torch.int32, (T, k))
    o = {} if out is None else out
    if not o:  # one allocation for the int32 outputs (five cost 12 us), pointers by offset
        n = T * k
        ints = _empty((n + E * C + 2 * E + 1,), torch.int32, expert_idx.device, stream)
        # ("unsafe" for autograd only: the parts are no views of one another to it)
        slot, o["tok_of_row"], o["arrivals"], o["kept_cnt"], o["n_dropped"] = \
            torch.unsafe_split_with_sizes(ints, (n, E * C, E, E, 1))
        o["slot"] = slot.view(T, k)
        o["kept"] = _empty((T, k), torch.uint8, expert_idx.device, stream)
        at = ints.data_ptr()
        _check(lib.moe_assign(ctypes.byref(cfg), ep, at, o["kept"].data_ptr(), at + 4 * n,
                              at + 4 * (n + E * C), at + 4 * (n + E * C + E),
                              at + 4 * (n + E * C + 2 * E), _status(status), _stream(stream)),
               "moe_assign")
        return o
    ptrs = []
    for name, dtype, shape in (("slot", torch.int32, (T, k)), ("kept", torch.uint8, (T, k)),
                               ("tok_of_row", torch.int32, (E * C,)),
                               ("arrivals", torch.int32, (E,)), ("kept_cnt", torch.int32, (E,)),
                               ("n_dropped", torch.int32, (1,))):
        if name not in o:
            o[name] = _empty(shape, dtype, expert_idx.device, stream)
        ptrs.append(_arg(o[name], name, dtype, shape))
    _check(lib.moe_assign(ctypes.byref(cfg), ep, *ptrs, _status(status), _stream(stream)),
           "moe_assign")
    return o


def dispatch_backward(cfg, dxe, expert_idx, slot, kept, dx=None, status=None, stream=None):
    """Gradient of ``dispatch``: dx [T, d] sums the kept choices' rows of dxe [E, C, d]."""
    T, act = cfg.T, _act_dtype(cfg)
    if dx is None:
        dx = _empty((T, cfg.d_model), act, dxe.device, stream)
    _check(lib.moe_dispatch_backward(
        ctypes.byref(cfg), _arg_rows(dxe, "dxe", act, (cfg.E, cfg.capacity, cfg.d_model)),
        *_choice_args(cfg, expert_idx, slot, kept), _arg(dx, "dx", act, (T, cfg.d_model)),
        _status(status), _stream(stream)), "moe_dispatch_backward")
    return dx


def combine_backward(cfg, dy, ye, expert_idx, gate, slot, kept, dye=None, dgate=None, status=None,
                     stream=None):
    """Gradients of ``combine``: (dye [E, C, d], dgate [T, k]).  Rows of ``dye`` that no token
    fills are left as they are (zeros in a ``dye`` made here); ``dye`` may be ``ye``."""
    T, k, act = cfg.T, cfg.k, _act_dtype(cfg)
    rows = (cfg.E, cfg.capacity, cfg.d_model)
    if dye is None:
        dye = _empty(rows, act, ye.device, stream)
        with torch.cuda.stream(stream):
            dye.zero_()
    if dgate is None:
        dgate = _empty((T, k), torch.float32, ye.device, stream)
    ep, sp, kp = _choice_args(cfg, expert_idx, slot, kept)
    _check(lib.moe_combine_backward(
        ctypes.byref(cfg), _arg(dy, "dy", act, (T, cfg.d_model)), _arg_rows(ye, "ye", act, rows), ep,
        _arg(gate, "gate", torch.float32, (T, k)), sp, kp, _arg_rows(dye, "dye", act, rows),
        _arg(dgate, "dgate", torch.float32, (T, k)), _status(status), _stream(stream)),
        "moe_combine_backward")
    return dye, dgate


def ffn_workspace_size(cfg: MoEConfig) -> int:
    config_check(cfg)
    return int(lib.moe_ffn_workspace_size(ctypes.byref(cfg)))


def set_wait_limit_ns(ns: int):
    """Limit of every bounded wait in the library's kernels (0 = the 1 s default)."""
    lib.moe_set_wait_limit_ns(int(ns))


def wait_limit_ns() -> int:
    return int(lib.moe_wait_limit_ns())


def expert_ffn(cfg, xe, W1, W2, kept_cnt, H=None, ye=None, workspace=None, status=None,
               stream=None, flags=0):
    """flags: FFN_WORKSPACE_ZEROED = the caller zeroed ``workspace`` on the stream already."""
    if H is None:
        H = torch.empty(cfg.E, cfg.capacity, cfg.d_ff, dtype=xe.dtype, device=xe.device)
    if ye is None:
        ye = torch.empty(cfg.E, cfg.capacity, cfg.d_model, dtype=xe.dtype, device=xe.device)
    if workspace is None:
        workspace = torch.empty(max(256, ffn_workspace_size(cfg)), dtype=torch.uint8,
                                device=xe.device)
    _check(lib.moe_expert_ffn_ex(ctypes.byref(cfg), _ptr(xe, "xe"), _ptr(W1, "W1"),
                                 _ptr(W2, "W2"), _ptr(kept_cnt, "kept_cnt"), _ptr(H, "H"),
                                 _ptr(ye, "ye"), _ptr(workspace, "workspace"), workspace.numel(),
                                 int(flags), _ptr(status, "status"), _stream(stream)),
           "moe_expert_ffn_ex")
    return H, ye


def combine(cfg, ye, expert_idx, gate, slot, kept, y=None, status=None, stream=None):
    if cfg.k > 2:
        act = _act_dtype(cfg)
        if y is None:
            y = _empty((cfg.T, cfg.d_model), act, ye.device, stream)
        ep, sp, kp = _choice_args(cfg, expert_idx, slot, kept)
        _check(lib.moe_combine(
            ctypes.byref(cfg), _arg_rows(ye, "ye", act, (cfg.E, cfg.capacity, cfg.d_model)), ep,
            _arg(gate, "gate", torch.float32, (cfg.T, cfg.k)), sp, kp,
            _arg(y, "y", act, (cfg.T, cfg.d_model)), _status(status), _stream(stream)),
            "moe_combine")
        return y
    if y is None:
        y = torch.empty(cfg.T, cfg.d_model, dtype=ye.dtype, device=ye.device)
    _check(lib.moe_combine(ctypes.byref(cfg), _ptr(ye, "ye"), _ptr(expert_idx, "expert_idx"),
                           _ptr(gate, "gate"), _ptr(slot, "slot"), _ptr(kept, "kept"),
                           _ptr(y, "y"), _ptr(status, "status"), _stream(stream)), "moe_combine")
    return y


def ep_ffn_config(cfg: MoEConfig, world: int) -> MoEConfig:
    """The expert-FFN config of one of ``world`` expert-parallel ranks:
    E / world experts, capacity world * C."""
    out = MoEConfig()
    _check(lib.moe_ep_ffn_config(ctypes.byref(cfg), int(world), ctypes.byref(out)),
           "moe_ep_ffn_config")
    return out


def _peer_table(peers, world, name):
    """Host array of ``world`` device addresses from tensors or ints (mapped peer pointers)."""
    if peers is None:
        return None
    if len(peers) != world:
        raise ValueError(f"{name} needs {world} entries, got {len(peers)}")
    addr = []
    for q, p in enumerate(peers):
        if isinstance(p, torch.Tensor):
            addr.append(_ptr(p, f"{name}[{q}]"))
        else:
            addr.append(int(p))
    return (ctypes.c_void_p * world)(*addr)


def ep_dispatch(cfg, rank, world, x, expert_idx, slot, kept, cnt_all, xe_peers, local_cnt=None,
                status=None, stream=None):
    """Expert-parallel dispatch: this rank's kept rows into their home ranks'
    receive buffers ``xe_peers`` (tensors or mapped device addresses, rank
    order).  Returns ``local_cnt`` [E / world], the rows each local expert
    receives from all ranks."""
    if local_cnt is None:
        local_cnt = torch.empty(cfg.E // world, dtype=torch.int32, device=cnt_all.device)
    _check(lib.moe_ep_dispatch(ctypes.byref(cfg), int(rank), int(world), _ptr(x, "x"),
                               _ptr(expert_idx, "expert_idx"), _ptr(slot, "slot"),
                               _ptr(kept, "kept"), _ptr(cnt_all, "cnt_all"),
                               _peer_table(xe_peers, world, "xe_peers"),
                               _ptr(local_cnt, "local_cnt"), _ptr(status, "status"),
                               _stream(stream)), "moe_ep_dispatch")
    return local_cnt


def ep_combine(cfg, rank, world, ye_peers, expert_idx, gate, slot, kept, cnt_all, y=None,
               status=None, stream=None):
    """Expert-parallel combine: y [T, d] from the home ranks' expert outputs
    ``ye_peers`` (tensors or mapped device addresses, rank order)."""
    if y is None:
        dt = torch.bfloat16 if cfg.dtype == DTYPE_BF16 else torch.float32
        y = torch.empty(cfg.T, cfg.d_model, dtype=dt, device=cnt_all.device)
    _check(lib.moe_ep_combine(ctypes.byref(cfg), int(rank), int(world),
                              _peer_table(ye_peers, world, "ye_peers"),
                              _ptr(expert_idx, "expert_idx"), _ptr(gate, "gate"),
                              _ptr(slot, "slot"), _ptr(kept, "kept"), _ptr(cnt_all, "cnt_all"),
                              _ptr(y, "y"), _ptr(status, "status"), _stream(stream)),
           "moe_ep_combine")
    return y


STAGES = ("router", "route_assign", "dispatch", "expert_ffn", "combine")


def layer_forward(cfg, x, W1, W2, *, Wr=None, bias=None, domain_id=None, y=None, workspace=None,
                  status=None, stream=None, stage_events=None):
    """The whole layer on the current stream.  Returns y; ``workspace`` keeps the intermediates.

    ``stage_events``: optional 6 ``torch.cuda.Event`` recorded before and after the
    stages named in ``STAGES`` (a profiling hook)."""
    if y is None:
        y = torch.empty(cfg.T, cfg.d_model, dtype=x.dtype, device=x.device)
    if workspace is None:
        workspace = torch.empty(workspace_size(cfg), dtype=torch.uint8, device=x.device)
    ev = None
    if stage_events is not None:
        if len(stage_events) != 6:
            raise ValueError("stage_events needs 6 events")
        s = stream if stream is not None else torch.cuda.current_stream()
        for e in stage_events:
            if e is not None and not e.cuda_event:
                e.record(s)  # torch creates its events lazily; the library re-records them
        ev = (ctypes.c_void_p * 6)(*[e.cuda_event if e is not None else None for e in stage_events])
    _check(lib.moe_layer_forward(ctypes.byref(cfg), _ptr(x, "x"), _ptr(Wr, "Wr"), _ptr(bias, "bias"),
                                 _ptr(domain_id, "domain_id"), _ptr(W1, "W1"), _ptr(W2, "W2"),
                                 _ptr(y, "y"), _ptr(workspace, "workspace"), workspace.numel(),
                                 _ptr(status, "status"),
                                 None if ev is None else ctypes.cast(ev, _vp), _stream(stream)),
           "moe_layer_forward")
    return y


def workspace_views(cfg, workspace) -> dict:
    """Tensor views of the intermediates moe_layer_forward leaves in its workspace."""
    m = workspace_layout(cfg)
    T, k, E, C, d, f = cfg.T, cfg.k, cfg.E, cfg.capacity, cfg.d_model, cfg.d_ff
    act = _act_dtype(cfg)
    es = 2 if act == torch.bfloat16 else 4

    def view(off, n, dtype, shape, itemsize):
        return workspace[off: off + n * itemsize].view(dtype).view(*shape)

    v = dict(
        expert_idx=view(m.expert_idx, T * k, torch.int32, (T, k), 4),
        gate=view(m.gate, T * k, torch.float32, (T, k), 4),
        slot=view(m.slot, T * k, torch.int32, (T, k), 4),
        kept=view(m.kept, T * k, torch.uint8, (T, k), 1),
        tok_of_row=view(m.tok_of_row, E * C, torch.int32, (E * C,), 4),
        arrivals=view(m.arrivals, E, torch.int32, (E,), 4),
        kept_cnt=view(m.kept_cnt, E, torch.int32, (E,), 4),
        n_dropped=view(m.n_dropped, 1, torch.int32, (1,), 4),
        xe=view(m.xe, E * C * d, act, (E, C, d), es),
        H=view(m.H, E * C * f, act, (E, C, f), es),
        ye=view(m.ye, E * C * d, act, (E, C, d), es),
    )
    if cfg.mode == ROUTE_TOPK and cfg.dtype == DTYPE_F32:  # bf16 layers keep no logits
        v["logits"] = view(m.logits, T * E, torch.float32, (T, E), 4)
    return v


def sparseclip_workspace_size(n_dense: int, n_sparse: int) -> int:
    return int(lib.sparseclip_workspace_size(n_dense, n_sparse))


def sparseclip_norm(dense, sparse, num_experts, out=None, workspace=None, stream=None):
    """SparseClip norm of lists of fp32 CUDA tensors; returns device double[3]
    = (norm, sum of squares dense, sum of squares expert)."""
    dense, sparse = list(dense), list(sparse)
    dev = (dense + sparse)[0].device
    if out is None:
        out = torch.empty(3, dtype=torch.float64, device=dev)
    if workspace is None:
        workspace = torch.empty(max(16, sparseclip_workspace_size(len(dense), len(sparse))),
                                dtype=torch.uint8, device=dev)

    def arrays(ts, name):
        ptrs = (ctypes.c_void_p * max(1, len(ts)))(*[_ptr(t, name) for t in ts])
        lens = (ctypes.c_int64 * max(1, len(ts)))(*[t.numel() for t in ts])
        return ptrs, lens

    for t in dense + sparse:
        if t.dtype != torch.float32:
            raise TypeError("SparseClip gradients must be fp32")
    dp, dl = arrays(dense, "dense")
    sp, sl = arrays(sparse, "sparse")
    _check(lib.sparseclip_norm(ctypes.cast(dp, _vp), ctypes.cast(dl, _vp), len(dense),
                               ctypes.cast(sp, _vp), ctypes.cast(sl, _vp), len(sparse),
                               num_experts, _ptr(out, "out"), _ptr(workspace, "workspace"),
                               workspace.numel(), _stream(stream)), "sparseclip_norm")
    return out


def sparseclip_clip(dense, sparse, num_experts, max_norm, out=None, workspace=None, stream=None):
    """SparseClip clipping of lists of fp32 CUDA tensors, in place; returns
    device double[4] = (norm before clipping, sum of squares dense, sum of
    squares expert, coef applied)."""
    dense, sparse = list(dense), list(sparse)
    dev = (dense + sparse)[0].device
    if out is None:
        out = torch.empty(4, dtype=torch.float64, device=dev)
    if workspace is None:
        workspace = torch.empty(max(16, sparseclip_workspace_size(len(dense), len(sparse))),
                                dtype=torch.uint8, device=dev)

    def arrays(ts, name):
        ptrs = (ctypes.c_void_p * max(1, len(ts)))(*[_ptr(t, name) for t in ts])
        lens = (ctypes.c_int64 * max(1, len(ts)))(*[t.numel() for t in ts])
        return ptrs, lens

    for t in dense + sparse:
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise TypeError("SparseClip gradients must be contiguous fp32")
    dp, dl = arrays(dense, "dense")
    sp, sl = arrays(sparse, "sparse")
    _check(lib.sparseclip_clip(ctypes.cast(dp, _vp), ctypes.cast(dl, _vp), len(dense),
                               ctypes.cast(sp, _vp), ctypes.cast(sl, _vp), len(sparse),
                               num_experts, float(max_norm), _ptr(out, "out"),
                               _ptr(workspace, "workspace"), workspace.numel(), _stream(stream)),
           "sparseclip_clip")
    return out


Q_BLOCK = 256  # elements of a tensor that share one scale of the 8-bit moments


def adamw_state(params, bits=32):
    """Zero moments for a list of fp32 parameters, as keyword arguments of ``adamw_tensors``:
    fp32 (bits=32), or e4m3 codes with one fp32 scale per 256 elements (bits=8)."""
    if bits not in (32, 8):
        raise ValueError("bits must be 32 or 8")

    def zeros(dtype, blocks=False):
        return [torch.zeros(-(-p.numel() // Q_BLOCK) if blocks else p.numel(), dtype=dtype,
                            device=p.device) for p in params]

    if bits == 32:
        return dict(exp_avg=zeros(torch.float32), exp_avg_sq=zeros(torch.float32))
    return dict(exp_avg=zeros(torch.float8_e4m3fn), exp_avg_sq=zeros(torch.float8_e4m3fn),
                exp_avg_scale=zeros(torch.float32, True),
                exp_avg_sq_scale=zeros(torch.float32, True))


class AdamWTensors:
    """The tensors of an AdamW step, checked and laid out once (``adamw_tensors``).  It holds
    on to the tensors; a step reads and writes the memory they had when it was made, the
    gradients' too.  Where a backward pass puts its gradients into new tensors, copy them into
    these or make a new layout: a step on this one would take the old gradients, without an
    error, since they are kept alive here."""

    def __init__(self, n, device, grad_dtype, bits, arrays, keep):
        self.n, self.device, self.grad_dtype, self.bits = n, device, grad_dtype, bits
        self.arrays, self.keep = arrays, keep


def adamw_tensors(params, grads, exp_avg, exp_avg_sq, *, exp_avg_scale=None,
                  exp_avg_sq_scale=None, bf16_copies=None) -> AdamWTensors:
    """Lists of tensors for ``adamw_step``: fp32 ``params``; ``grads`` all fp32 or all bf16;
    the moments fp32, or float8_e4m3fn with their fp32 scales (one per 256 elements);
    ``bf16_copies`` (optional, entries may be None) receive the new parameters in bf16.  All
    contiguous, on one device, with the parameter's number of elements; nothing that the
    step writes may overlap anything else.

    For buffers that stay where they are over the training (gradients zeroed or overwritten in
    place, not set to None): the checks cost 3 to 7 us a tensor once, and the steps nothing."""
    params, grads = list(params), list(grads)
    n = len(params)
    dev = params[0].device if n else None
    gdt = grads[0].dtype if grads else torch.float32
    exp_avg, exp_avg_sq = list(exp_avg), list(exp_avg_sq)
    bits = 8 if exp_avg and exp_avg[0].dtype == torch.float8_e4m3fn else 32
    if bits == 8 and (exp_avg_scale is None or exp_avg_sq_scale is None):
        raise ValueError("8-bit moments need exp_avg_scale and exp_avg_sq_scale")
    sdt = torch.float8_e4m3fn if bits == 8 else torch.float32
    numel = [p.numel() for p in params]
    blocks = [-(-m // Q_BLOCK) for m in numel]

    def pointers(ts, name, dtype, sizes, optional=False):
        ts = list(ts)
        if len(ts) != n:
            raise ValueError(f"{name} needs {n} entries, got {len(ts)}")
        out = (ctypes.c_void_p * max(1, n))()
        for i, t in enumerate(ts):
            if t is None and optional:
                continue
            if t.dtype != dtype:
                raise TypeError(f"{name}[{i}] must be {dtype}, got {t.dtype}")
            if t.numel() != sizes[i]:
                raise ValueError(f"{name}[{i}] must have {sizes[i]} elements, got {t.numel()}")
            if t.device != dev:
                raise ValueError(f"{name}[{i}] is on {t.device}, params[0] on {dev}")
            out[i] = _ptr(t, f"{name}[{i}]")
        return out, ts

    made = [pointers(params, "params", torch.float32, numel),
            pointers(grads, "grads", gdt, numel),
            pointers(exp_avg, "exp_avg", sdt, numel),
            pointers(exp_avg_sq, "exp_avg_sq", sdt, numel)]
    made += ([pointers(exp_avg_scale, "exp_avg_scale", torch.float32, blocks),
              pointers(exp_avg_sq_scale, "exp_avg_sq_scale", torch.float32, blocks)]
             if bits == 8 else [(None, None), (None, None)])
    made.append((None, None) if bf16_copies is None else
                pointers(bf16_copies, "bf16_copies", torch.bfloat16, numel, optional=True))
    lens = (ctypes.c_int64 * max(1, n))(*numel)
    arrays = [ctypes.cast(lens, _vp)] + [None if a is None else ctypes.cast(a, _vp)
                                         for a, _ in made]
    cfg = AdamWConfig(grad_dtype=_dtype_code(gdt), state_bits=bits)
    _check(lib.moe_adamw_check(ctypes.byref(cfg), n, *arrays), "moe_adamw_check")
    return AdamWTensors(n, dev, cfg.grad_dtype, bits, arrays, (lens, made))


def adamw_step(tensors, *, step=1, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2,
               norm=None, max_norm=0.0, step_lr=None, status=None, stream=None):
    """One AdamW step over ``tensors`` (``adamw_tensors``), in place.

    ``norm``: float64 device tensor whose first element is the gradients' norm (the output of
    ``sparseclip_norm``); the gradients are scaled by min(1, max_norm / norm) as they are read.
    ``step_lr``: float64 device tensor (step, lr) read instead of ``step`` and ``lr``, for a
    step captured into a CUDA graph."""
    if tensors.n and tensors.device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {tensors.device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    np_ = None if norm is None else _arg(norm, "norm", torch.float64, norm.shape)
    sp = None if step_lr is None else _arg(step_lr, "step_lr", torch.float64, (2,))
    if norm is not None and norm.numel() < 1:
        raise ValueError("norm is empty")
    cfg = AdamWConfig(lr=lr, beta1=betas[0], beta2=betas[1], eps=eps, weight_decay=weight_decay,
                      max_norm=max_norm, step=step, grad_dtype=tensors.grad_dtype,
                      state_bits=tensors.bits)
    _check(lib.moe_adamw_step(ctypes.byref(cfg), tensors.n, *tensors.arrays, np_, sp,
                              _status(status), _stream(stream)), "moe_adamw_step")
