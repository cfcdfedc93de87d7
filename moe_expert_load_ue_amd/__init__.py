"""Python binding of libue, the MI355X (gfx950) per-layer MoE expert
rebalancing library (C ABI in ``include/ue.h``).

Argument marshalling only: every step of the path runs in the HIP kernels
behind the C ABI. PyTorch provides device memory and streams. The binding
raises at import of the first call if ``libue.so`` is not built; there is no
fallback implementation.

Functions carry the C names (``ue_load``, ``ue_plan``, ``ue_reroute``,
``ue_rebalance``,
``ue_weight_sync``, ``ue_grad_reduce``, ``ue_gather_rows``, ...) and take a
:class:`Context` plus torch tensors; :class:`Context` also exposes them as
methods without the prefix.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libue.so")

UE_OK = 0
STATUS = {0: "UE_OK", -1: "UE_EINVAL", -2: "UE_ESHAPE", -3: "UE_ENOMEM",
          -4: "UE_EHIP", -5: "UE_EUNSUPPORTED", -6: "UE_ESTATE"}


class UEError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class ue_config(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32),
                ("num_ranks", ctypes.c_int32),
                ("spare_per_rank", ctypes.c_int32),
                ("topk", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32),
                ("max_layers", ctypes.c_int32),
                ("plan_policy", ctypes.c_int32),
                ("quota_mode", ctypes.c_int32)]

PLAN_LEAST_LOADED, PLAN_BEST_FIT, PLAN_BEST_FIT_COVER, PLAN_BEST_FIT_ASCENDING = \
    0, 1, 2, 3
QUOTA_FIXED, QUOTA_SEARCH = 0, 1


PLACEMENT_FIELDS = ("words", "quota", "exhausted", "residual", "n_rep",
                    "rep_off", "rep_slot", "rep_cap", "slot_expert",
                    "slot_cap", "slot_off", "load_before", "load_after")


class ue_placement_layout(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in PLACEMENT_FIELDS]


# Every symbol the header declares, with its ctypes signature.
_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
_f32 = ctypes.c_float

F32, BF16, I8 = 0, 1, 2
_TYPES = {torch.float32: F32, torch.bfloat16: BF16}
SCORES = {"softmax": 0, "sigmoid": 1}


class ue_i8_product(ctypes.Structure):
    _fields_ = ([(f, _vp) for f in ("a", "a_scale", "w", "w_scale", "offsets",
                                    "expert_of", "index", "out")] +
                [(f, _i64) for f in ("lda", "ldw", "w_stride", "ws_stride",
                                     "ldo")] +
                [(f, _i32) for f in ("a_rows", "n_mats", "groups", "index_div",
                                     "M", "N", "K", "gated", "out_type")])


class ue_weight_grad_product(ctypes.Structure):
    _fields_ = ([(f, _vp) for f in ("dy", "x", "x_scale", "offsets", "index",
                                    "out", "workspace")] +
                [(f, _i64) for f in ("lddy", "ldx", "lds", "ldo",
                                     "out_stride")] +
                [(f, _i32) for f in ("x_rows", "groups", "index_div", "M", "N",
                                     "K", "accumulate")])


class ue_layer(ctypes.Structure):
    _fields_ = ([(f, _vp) for f in ("router", "bias", "gate_up", "down",
                                    "gate_up_scale", "down_scale")] +
                [(f, _i64) for f in ("gate_up_stride", "down_stride")] +
                [(f, _i32) for f in ("hidden", "inter", "weight_type",
                                     "score", "renorm")] +
                [("scale", _f32)])


SIGNATURES = {
    "ue_create": (ctypes.c_int, [ctypes.POINTER(ue_config),
                                 ctypes.POINTER(_vp)]),
    "ue_destroy": (None, [_vp]),
    "ue_last_error": (ctypes.c_char_p, [_vp]),
    "ue_status_name": (ctypes.c_char_p, [ctypes.c_int]),
    "ue_get_placement_layout": (ctypes.c_int,
                                [_vp, ctypes.POINTER(ue_placement_layout)]),
    "ue_placement_bytes": (ctypes.c_size_t, [_vp]),
    "ue_load": (ctypes.c_int, [_vp, _vp, _i32, _i32, _vp, _vp, _vp]),
    "ue_plan": (ctypes.c_int, [_vp, _vp, _i32, _vp, _vp]),
    "ue_reroute": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp,
                                  _vp, _vp, _vp]),
    "ue_rebalance": (ctypes.c_int, [_vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp,
                                    _vp, _vp, _vp, _vp, _vp]),
    "ue_set_timing": (ctypes.c_int, [_vp, ctypes.c_int]),
    "ue_kernel_times": (ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_float),
                                       _i32, ctypes.POINTER(_i32)]),
    "ue_register_experts": (ctypes.c_int, [_vp, _i32, _i32,
                                           ctypes.POINTER(_i64),
                                           ctypes.POINTER(_vp),
                                           ctypes.POINTER(_vp), _i32,
                                           ctypes.POINTER(_vp),
                                           ctypes.POINTER(_vp)]),
    "ue_weight_sync": (ctypes.c_int, [_vp, _vp, _vp, _i32, _vp]),
    "ue_grad_reduce": (ctypes.c_int, [_vp, _vp, _vp, _i32, _vp]),
    "ue_gather_rows": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _i32, _vp,
                                      _vp]),
    "ue_stale_loads": (ctypes.c_int, [_vp, _vp, _vp, _i32, _vp, _vp]),
    "ue_set_wait_limit": (ctypes.c_int, [_vp, ctypes.c_uint32]),
    "ue_gate": (ctypes.c_int, [_vp, _vp, _i32, _i64, _i32, _i32, _i32, _f32,
                               _vp, _vp, _vp, _vp]),
    "ue_gate_backward": (ctypes.c_int, [_vp, _vp, _i32, _i64, _i32, _i32,
                                        _i32, _f32, _vp, _vp, _vp, _i64,
                                        _vp]),
    "ue_quantize_rows": (ctypes.c_int, [_vp, _vp, _i32, _i64, _i32, _i32, _vp,
                                        _i64, _vp, _vp]),
    "ue_matmul_i8": (ctypes.c_int, [_vp, _vp, _vp]),
    "ue_register_layer": (ctypes.c_int, [_vp, ctypes.POINTER(ue_layer)]),
    "ue_moe_tokens": (ctypes.c_int, [_vp, _vp, _i64, _i32, _vp, _i64, _vp,
                                     _vp, _vp]),
    "ue_balance_workspace": (ctypes.c_size_t, [_vp, _i32, _i32]),
    "ue_balance": (ctypes.c_int, [_vp, _vp, _i32, _i64, _i32, _i32, _vp, _vp,
                                  _i32, _vp, _vp, _vp, _vp, _vp]),
    "ue_balance_backward": (ctypes.c_int, [_vp, _vp, _i32, _i64, _i32, _i32,
                                           _vp, _i32, _vp, _vp, _vp, _i64,
                                           _i32, _vp]),
    "ue_pack_rows": (ctypes.c_int, [_vp, _vp, _i32, _i64, _i32, _i32, _vp,
                                    _i64, _vp, _i64, _vp]),
    "ue_unpack_rows": (ctypes.c_int, [_vp, _vp, _i64, _vp, _i64, _i32, _i32,
                                      _vp, _i32, _i64, _vp]),
    "ue_gated": (ctypes.c_int, [_vp, _vp, _i32, _i64, _i32, _i32, _vp, _i64,
                                _vp, _i64, _vp, _i64, _vp]),
    "ue_gated_backward": (ctypes.c_int, [_vp, _vp, _i64, _vp, _i64, _vp, _i32,
                                         _i64, _i32, _i32, _vp, _i64, _vp,
                                         _i64, _vp]),
    "ue_weight_grad_workspace": (ctypes.c_size_t, [_vp, _vp]),
    "ue_weight_grad": (ctypes.c_int, [_vp, _vp, _vp]),
    "ue_combine": (ctypes.c_int, [_vp, _vp, _i32, _i64, _i32, _vp, _vp, _vp,
                                  _i64, _i32, _i32, _vp, _i64, _vp]),
    "ue_combine_backward": (ctypes.c_int, [_vp, _vp, _i32, _i64, _vp, _vp, _vp,
                                           _i64, _i32, _i32, _i32, _vp, _i64,
                                           _vp, _vp]),
    "ue_combine_backward_workspace": (ctypes.c_size_t, [_vp, _i32, _i32]),
    "ue_combine_backward_all": (ctypes.c_int, [_vp, _vp, _i32, _i64, _vp, _vp,
                                               _vp, _i64, _i32, _i32, _i32,
                                               _vp, _i64, _vp, _vp, _vp]),
    "ue_rebalance_static": (ctypes.c_int, [ctypes.POINTER(ue_config), _vp,
                                           _i32, _i32, _vp, _vp, _vp, _vp,
                                           _vp, _vp, _vp, _vp, _vp]),
}

_lib = None


def library():
    """The loaded libue.so (raises if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run "
                "`python -m moe_expert_load_ue_amd.build` (hipcc, gfx950)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name, dtype, device, numel=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} elements, has {t.numel()}")
    return t


class Context:
    """One ``ue_ctx`` on one device (see ``ue_create`` in ``ue.h``)."""

    def __init__(self, num_experts: int, num_ranks: int, spare_per_rank: int,
                 topk: int, max_tokens: int, max_layers: int = 1,
                 device=None, plan_policy: int = PLAN_LEAST_LOADED,
                 quota_mode: int = QUOTA_FIXED):
        self.device = torch.device(device if device is not None else
                                   f"cuda:{torch.cuda.current_device()}")
        self.E, self.R, self.S = int(num_experts), int(num_ranks), int(
            spare_per_rank)
        self.k, self.max_tokens = int(topk), int(max_tokens)
        self.max_layers = int(max_layers)
        self.plan_policy = int(plan_policy)
        self.quota_mode = int(quota_mode)
        self.N = self.E // self.R if self.R else 0
        self.P = self.R * (self.N + self.S)
        cfg = ue_config(self.E, self.R, self.S, self.k, self.max_tokens,
                        self.max_layers, self.plan_policy, self.quota_mode)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            rc = library().ue_create(ctypes.byref(cfg), ctypes.byref(h))
        if rc != UE_OK:
            raise UEError(rc, "ue_create refused the configuration")
        self._h = h
        self._index = (self.device.index if self.device.index is not None
                       else torch.cuda.current_device())
        lay = ue_placement_layout()
        library().ue_get_placement_layout(self._h, ctypes.byref(lay))
        self.layout = {f: getattr(lay, f) for f in PLACEMENT_FIELDS}
        self.placement_words = lay.words
        self._registered = None
        self.hidden = None          # of the registered layer

    # -- lifetime ----------------------------------------------------------
    def close(self):
        if getattr(self, "_h", None):
            library().ue_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, rc, what):
        if rc != UE_OK:
            msg = library().ue_last_error(self._h).decode()
            raise UEError(rc, f"{what}: {msg}")

    # -- placement helpers --------------------------------------------------
    def new_placement(self, L: int) -> torch.Tensor:
        return torch.empty((L, self.placement_words), dtype=torch.int32,
                           device=self.device)

    def placement_fields(self, placement: torch.Tensor) -> dict:
        """Views of one or more placement blocks by field name."""
        pl = placement.reshape(-1, self.placement_words)
        lay, E, P, R = self.layout, self.E, self.P, self.R
        sizes = dict(rep_off=E + 1, rep_slot=P, rep_cap=P, slot_expert=P,
                     slot_cap=P, slot_off=P + 1, load_before=R, load_after=R)
        out = {k: pl[:, lay[k]] for k in ("quota", "exhausted", "residual",
                                          "n_rep")}
        for k, n in sizes.items():
            out[k] = pl[:, lay[k]:lay[k] + n]
        return out

    # -- steps (methods mirror the module-level functions) ------------------
    def load(self, routing, counts=None, invalid=None, stream=None):
        return ue_load(self, routing, counts, invalid, stream)

    def plan(self, counts, placement=None, stream=None):
        return ue_plan(self, counts, placement, stream)

    def reroute(self, routing, placement, **kw):
        return ue_reroute(self, routing, placement, **kw)

    def rebalance(self, routing, **kw):
        return ue_rebalance(self, routing, **kw)

    def register_experts(self, *a, **kw):
        return ue_register_experts(self, *a, **kw)

    def weight_sync(self, rep_off, rep_buf, n_experts=None, stream=None):
        return ue_weight_sync(self, rep_off, rep_buf, n_experts, stream)

    def grad_reduce(self, rep_off, rep_buf, n_experts=None, stream=None):
        return ue_grad_reduce(self, rep_off, rep_buf, n_experts, stream)

    def gather_rows(self, x, inv_perm, out=None, stream=None):
        return ue_gather_rows(self, x, inv_perm, out, stream)

    def gate(self, logits, **kw):
        return ue_gate(self, logits, **kw)

    def gate_backward(self, logits, ids, dweights, **kw):
        return ue_gate_backward(self, logits, ids, dweights, **kw)

    def quantize_rows(self, x, **kw):
        return ue_quantize_rows(self, x, **kw)

    def matmul_i8(self, a, a_scale, w, w_scale, **kw):
        return ue_matmul_i8(self, a, a_scale, w, w_scale, **kw)

    def register_layer(self, router, gate_up, down, *scales, **kw):
        return ue_register_layer(self, router, gate_up, down, *scales, **kw)

    def moe_tokens(self, x, **kw):
        return ue_moe_tokens(self, x, **kw)

    def balance(self, logits, ids, offsets=None, **kw):
        return ue_balance(self, logits, ids, offsets, **kw)

    def balance_backward(self, logits, counts, dloss, offsets=None, **kw):
        return ue_balance_backward(self, logits, counts, dloss, offsets, **kw)

    def pack_rows(self, x, **kw):
        return ue_pack_rows(self, x, **kw)

    def unpack_rows(self, q, scale, **kw):
        return ue_unpack_rows(self, q, scale, **kw)

    def gated(self, gu, **kw):
        return ue_gated(self, gu, **kw)

    def gated_backward(self, dh, q, scale, **kw):
        return ue_gated_backward(self, dh, q, scale, **kw)

    def weight_grad(self, dy, x, x_scale=None, **kw):
        return ue_weight_grad(self, dy, x, x_scale, **kw)

    def combine(self, y, inv_perm, weights=None, **kw):
        return ue_combine(self, y, inv_perm, weights, **kw)

    def combine_backward(self, dout, inv_perm, weights=None, **kw):
        return ue_combine_backward(self, dout, inv_perm, weights, **kw)


def ue_create(num_experts, num_ranks, spare_per_rank, topk, max_tokens,
              max_layers=1, device=None, plan_policy=PLAN_LEAST_LOADED,
              quota_mode=QUOTA_FIXED) -> Context:
    return Context(num_experts, num_ranks, spare_per_rank, topk, max_tokens,
                   max_layers, device, plan_policy, quota_mode)


def ue_destroy(ctx: Context):
    ctx.close()


def ue_placement_bytes(ctx: Context) -> int:
    return int(library().ue_placement_bytes(ctx._h))


def ue_get_placement_layout(ctx: Context) -> dict:
    return dict(ctx.layout)


def ue_last_error(ctx: Context) -> str:
    return library().ue_last_error(ctx._h).decode()


def _routing_shape(ctx, routing):
    if routing.dim() == 2:
        routing = routing.unsqueeze(0)
    if routing.dim() != 3 or routing.shape[2] != ctx.k:
        raise ValueError(f"routing must be [L, T, {ctx.k}]")
    return routing, routing.shape[0], routing.shape[1]


def ue_load(ctx: Context, routing, counts=None, invalid=None, stream=None):
    """counts int32 [L, E] of routing int32 [L, T, k]."""
    routing, L, T = _routing_shape(ctx, routing)
    _need(routing, "routing", torch.int32, ctx.device)
    if counts is None:
        counts = torch.empty((L, ctx.E), dtype=torch.int32, device=ctx.device)
    _need(counts, "counts", torch.int32, ctx.device, L * ctx.E)
    if invalid is not None:
        _need(invalid, "invalid", torch.int32, ctx.device, L)
    rc = library().ue_load(ctx._h, _ptr(routing), L, T, _ptr(counts),
                           _ptr(invalid), _stream(stream, ctx.device))
    ctx._check(rc, "ue_load")
    return counts


def ue_plan(ctx: Context, counts, placement=None, stream=None):
    """Placement blocks int32 [L, words] from counts int32 [L, E]."""
    counts = counts.reshape(-1, ctx.E)
    L = counts.shape[0]
    _need(counts, "counts", torch.int32, ctx.device)
    if placement is None:
        placement = ctx.new_placement(L)
    _need(placement, "placement", torch.int32, ctx.device,
          L * ctx.placement_words)
    rc = library().ue_plan(ctx._h, _ptr(counts), L, _ptr(placement),
                           _stream(stream, ctx.device))
    ctx._check(rc, "ue_plan")
    return placement


def ue_stale_loads(ctx: Context, placement, counts, rank_loads=None,
                   stream=None):
    """Rank loads int32 [L, R] when placement blocks made from earlier counts
    are applied to new counts int32 [L, E]."""
    counts = counts.reshape(-1, ctx.E)
    L = counts.shape[0]
    _need(counts, "counts", torch.int32, ctx.device)
    _need(placement, "placement", torch.int32, ctx.device,
          L * ctx.placement_words)
    if rank_loads is None:
        rank_loads = torch.empty((L, ctx.R), dtype=torch.int32,
                                 device=ctx.device)
    _need(rank_loads, "rank_loads", torch.int32, ctx.device, L * ctx.R)
    rc = library().ue_stale_loads(ctx._h, _ptr(placement), _ptr(counts), L,
                                  _ptr(rank_loads),
                                  _stream(stream, ctx.device))
    ctx._check(rc, "ue_stale_loads")
    return rank_loads


def ue_reroute(ctx: Context, routing, placement, phys=None, rank_counts=None,
               perm=None, inv_perm=None, faults=None, with_inv=True,
               stream=None):
    """Physical routing, per-rank counts, dispatch permutation (and its
    inverse) for every layer. Returns a dict of the output tensors."""
    routing, L, T = _routing_shape(ctx, routing)
    _need(routing, "routing", torch.int32, ctx.device)
    _need(placement, "placement", torch.int32, ctx.device,
          L * ctx.placement_words)
    A = T * ctx.k
    dev = ctx.device

    def mk(t, shape, name, need=True):
        if t is None and need:
            t = torch.empty(shape, dtype=torch.int32, device=dev)
        if t is not None:
            n = 1
            for s in shape:
                n *= s
            _need(t, name, torch.int32, dev, n)
        return t

    phys = mk(phys, (L, T, ctx.k), "phys")
    rank_counts = mk(rank_counts, (L, ctx.R), "rank_counts")
    perm = mk(perm, (L, A), "perm")
    inv_perm = mk(inv_perm, (L, A), "inv_perm", with_inv)
    faults = mk(faults, (L,), "faults")
    rc = library().ue_reroute(ctx._h, _ptr(routing), _ptr(placement), L, T,
                              _ptr(phys), _ptr(rank_counts), _ptr(perm),
                              _ptr(inv_perm), _ptr(faults),
                              _stream(stream, dev))
    ctx._check(rc, "ue_reroute")
    return dict(phys=phys, rank_counts=rank_counts, perm=perm,
                inv_perm=inv_perm, faults=faults)


POISONED = 0x40000000   # bit of invalid / faults: a wait gave up


def ue_set_wait_limit(ctx: Context, polls: int):
    """Polls one cross-workgroup wait may take before it gives up (0: at
    once, marking every multi-group layer poisoned)."""
    ctx._check(library().ue_set_wait_limit(ctx._h, int(polls)),
               "ue_set_wait_limit")


def ue_set_timing(ctx: Context, enable: bool = True):
    ctx._check(library().ue_set_timing(ctx._h, int(bool(enable))),
               "ue_set_timing")


def ue_kernel_times(ctx: Context) -> list:
    """Durations (ms) of the kernels of the latest timed call."""
    ms = (ctypes.c_float * 8)()
    n = ctypes.c_int32()
    ctx._check(library().ue_kernel_times(ctx._h, ms, 8, ctypes.byref(n)),
               "ue_kernel_times")
    return [ms[i] for i in range(n.value)]


def ue_rebalance(ctx: Context, routing, counts=None, invalid=None,
                 placement=None, phys=None, rank_counts=None, perm=None,
                 inv_perm=None, faults=None, with_inv=True, stream=None):
    """load -> plan -> reroute in one call (see ``ue_rebalance`` in ue.h).
    Returns a dict with every output tensor."""
    routing, L, T = _routing_shape(ctx, routing)
    _need(routing, "routing", torch.int32, ctx.device)
    A = T * ctx.k
    dev = ctx.device

    def mk(t, shape, name, need=True):
        if t is None and need:
            t = torch.empty(shape, dtype=torch.int32, device=dev)
        if t is not None:
            n = 1
            for s in shape:
                n *= s
            _need(t, name, torch.int32, dev, n)
        return t

    counts = mk(counts, (L, ctx.E), "counts")
    invalid = mk(invalid, (L,), "invalid")
    placement = mk(placement, (L, ctx.placement_words), "placement")
    phys = mk(phys, (L, T, ctx.k), "phys")
    rank_counts = mk(rank_counts, (L, ctx.R), "rank_counts")
    perm = mk(perm, (L, A), "perm")
    inv_perm = mk(inv_perm, (L, A), "inv_perm", with_inv)
    faults = mk(faults, (L,), "faults")
    rc = library().ue_rebalance(ctx._h, _ptr(routing), L, T, _ptr(counts),
                                _ptr(invalid), _ptr(placement), _ptr(phys),
                                _ptr(rank_counts), _ptr(perm), _ptr(inv_perm),
                                _ptr(faults), _stream(stream, dev))
    ctx._check(rc, "ue_rebalance")
    return dict(counts=counts, invalid=invalid, placement=placement,
                phys=phys, rank_counts=rank_counts, perm=perm,
                inv_perm=inv_perm, faults=faults)


STATIC_SCRATCH_BYTES = 16 << 20


def placement_words(num_experts, num_ranks, spare_per_rank):
    """int32 words of one layer's placement block for a configuration (the
    layout ue_get_placement_layout reports, padded to 64 words)."""
    E, R = int(num_experts), int(num_ranks)
    P = R * (E // R + int(spare_per_rank))
    return (6 + E + 5 * P + 2 * R + 63) // 64 * 64


def ue_rebalance_static(cfg: ue_config, routing, counts, invalid, placement,
                        phys, rank_counts, perm, inv_perm, faults,
                        stream=None):
    """ue_rebalance with no context and no allocation (see
    ``ue_rebalance_static`` in ue.h): every output is the caller's
    preallocated tensor (invalid and inv_perm may be None)."""
    if not isinstance(cfg, ue_config):
        raise TypeError("cfg must be a ue_config")
    if routing.dim() == 2:
        routing = routing.unsqueeze(0)
    L, T, k = routing.shape
    if k != cfg.topk:
        raise ValueError(f"routing has {k} experts per token, cfg {cfg.topk}")
    dev = routing.device
    _need(routing, "routing", torch.int32, dev)
    A = T * k
    words = placement_words(cfg.num_experts, cfg.num_ranks,
                            cfg.spare_per_rank)
    for t, name, n in ((counts, "counts", L * cfg.num_experts),
                       (invalid, "invalid", L),
                       (placement, "placement", L * words),
                       (phys, "phys", L * A),
                       (rank_counts, "rank_counts", L * cfg.num_ranks),
                       (perm, "perm", L * A), (inv_perm, "inv_perm", L * A),
                       (faults, "faults", L)):
        if t is not None or name not in ("invalid", "inv_perm"):
            _need(t, name, torch.int32, dev, n)
    rc = library().ue_rebalance_static(
        ctypes.byref(cfg), _ptr(routing), L, T, _ptr(counts), _ptr(invalid),
        _ptr(placement), _ptr(phys), _ptr(rank_counts), _ptr(perm),
        _ptr(inv_perm), _ptr(faults), _stream(stream, dev))
    if rc != UE_OK:
        raise UEError(rc, library().ue_last_error(None).decode())


def ue_register_experts(ctx: Context, mat_elems, master_w=None, master_g=None,
                        spare_w=None, spare_g=None):
    """Registers expert state. ``master_w[e][m]`` etc. are tensors (bf16
    weights, fp32 gradients), or None for the kind not registered.
    ``mat_elems[m]`` is the element count of matrix m."""
    n_mats = len(mat_elems)
    n_exp = len(master_w if master_w is not None else master_g)
    sp = spare_w if spare_w is not None else spare_g
    n_buf = len(sp) if sp is not None else 0

    def table(rows, dtype):
        if rows is None:
            return None
        arr = (ctypes.c_void_p * (len(rows) * n_mats))()
        for i, row in enumerate(rows):
            if len(row) != n_mats:
                raise ValueError("every expert needs one tensor per matrix")
            for m, t in enumerate(row):
                _need(t, "expert tensor", dtype, ctx.device, mat_elems[m])
                arr[i * n_mats + m] = t.data_ptr()
        return arr

    tw, tg = table(master_w, torch.bfloat16), table(master_g, torch.float32)
    sw, sg = table(spare_w, torch.bfloat16), table(spare_g, torch.float32)
    elems = (ctypes.c_int64 * n_mats)(*[int(v) for v in mat_elems])
    rc = library().ue_register_experts(ctx._h, n_exp, n_mats, elems, tw, tg,
                                       n_buf, sw, sg)
    ctx._check(rc, "ue_register_experts")
    # keep the tensors alive while the library holds their pointers
    ctx._registered = (master_w, master_g, spare_w, spare_g)


def _csr(ctx, rep_off, rep_buf, n_experts):
    _need(rep_off, "rep_off", torch.int32, ctx.device)
    _need(rep_buf, "rep_buf", torch.int32, ctx.device)
    n = rep_off.numel() - 1 if n_experts is None else int(n_experts)
    return n


def ue_weight_sync(ctx: Context, rep_off, rep_buf, n_experts=None,
                   stream=None):
    n = _csr(ctx, rep_off, rep_buf, n_experts)
    rc = library().ue_weight_sync(ctx._h, _ptr(rep_off), _ptr(rep_buf), n,
                                  _stream(stream, ctx.device))
    ctx._check(rc, "ue_weight_sync")


def ue_grad_reduce(ctx: Context, rep_off, rep_buf, n_experts=None,
                   stream=None):
    n = _csr(ctx, rep_off, rep_buf, n_experts)
    rc = library().ue_grad_reduce(ctx._h, _ptr(rep_off), _ptr(rep_buf), n,
                                  _stream(stream, ctx.device))
    ctx._check(rc, "ue_grad_reduce")


def replica_table(ctx: Context, placement, layer: int = 0):
    """The replica table of one layer's placement block as the (rep_off,
    rep_buf) pair that ue_weight_sync and ue_grad_reduce take: views of the
    block's rep_off and rep_slot fields, on the device. With one buffer
    registered per physical slot (buffer p for slot p), the plan drives the
    sync and the reduction directly."""
    blk = placement.reshape(-1, ctx.placement_words)[layer]
    lay = ctx.layout
    return (blk[lay["rep_off"]:lay["rep_off"] + ctx.E + 1],
            blk[lay["rep_slot"]:lay["rep_slot"] + ctx.P])


def ue_gather_rows(ctx: Context, x, inv_perm, out=None, stream=None):
    """out[pos] = x[perm[pos] // k] for one layer's inverse permutation."""
    if x.dim() != 2:
        raise ValueError("x must be [T, H]")
    T, H = x.shape
    _need(x, "x", torch.bfloat16, ctx.device)
    _need(inv_perm, "inv_perm", torch.int32, ctx.device, T * ctx.k)
    if out is None:
        out = torch.empty((T * ctx.k, H), dtype=torch.bfloat16,
                          device=ctx.device)
    _need(out, "out", torch.bfloat16, ctx.device, T * ctx.k * H)
    rc = library().ue_gather_rows(ctx._h, _ptr(x), _ptr(inv_perm), T, ctx.k,
                                  H, _ptr(out), _stream(stream, ctx.device))
    ctx._check(rc, "ue_gather_rows")
    return out


# ---- the expert layer around a rebalance ----------------------------------
# These calls also serve single tokens, where the time on the host counts:
# arguments are checked with few attribute reads and passed as plain integers.

_FLOATS = (torch.float32, torch.bfloat16)
_raw_stream = torch._C._cuda_getCurrentRawStream \
    if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _rows(t, name, device, types, cols=None):
    """A matrix [rows, cols] whose rows are contiguous; returns (rows, cols,
    distance between rows in elements)."""
    try:
        n, c = t.shape
        if t.dtype in types and t.device == device and (c == cols or
                                                        cols is None):
            ld, one = t.stride()
            if one == 1 or c <= 1:
                # a single row has no distance to the next: one that meets
                # every call
                return n, c, ld if n > 1 else (c + 15) // 16 * 16
    except (AttributeError, TypeError, ValueError):
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in types:
        raise TypeError(f"{name} must be one of {list(types)}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dim() != 2 or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} must be [rows, {cols or 'cols'}], is "
                         f"{tuple(t.shape)}")
    raise ValueError(f"{name} must have contiguous rows")


def _flat(t, name, dtype, device, numel):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or \
            t.device != device or t.numel() != numel or not t.is_contiguous():
        _need(t, name, dtype, device, numel)
    return t.data_ptr()


_device = torch._C._cuda_getDevice \
    if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


# Makes an uninitialised tensor on the current device: what generated code of
# torch.compile calls, 0.8 us on the host where torch.empty takes 1.7, of the 10
# that a call with three outputs took. It goes past torch's dispatcher, so it is
# taken only where that has nothing to do: no dispatch or function mode is on, and
# none but ordinary memory is asked for (deterministic mode fills it).
def _torch(*path):
    at = torch._C
    for name in path:
        at = getattr(at, name, None)
    return at


_empty = _torch("_dynamo", "guards", "_empty_strided_cuda")
_dispatch_modes = _torch("_len_torch_dispatch_stack")
_function_modes = _torch("_len_torch_function_stack")
_deterministic = _torch("_get_deterministic_algorithms")
if None in (_dispatch_modes, _function_modes, _deterministic):
    _empty = None


def _short(shape, dtype):
    dims = len(shape)
    if dims == 2:
        return _empty(shape, (shape[1] or 1, 1), dtype)
    if dims == 1:
        return _empty(shape, (1,), dtype)
    cols = shape[2] or 1
    return _empty(shape, ((shape[1] or 1) * cols, cols, 1), dtype)


def _maker(ctx, stream):
    """What makes a call's output tensors, whose memory belongs to the stream
    that writes them: f(shape, dtype). (Looking costs 0.25 us, so calls of
    several outputs look once.)"""
    if stream is None and _empty is not None and _device() == ctx._index and \
            not (_dispatch_modes() or _function_modes() or _deterministic()):
        return _short

    def make(shape, dtype):
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=ctx.device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=ctx.device)
    return make


def _new(shape, dtype, ctx, stream):
    return _maker(ctx, stream)(shape, dtype)


def _on(ctx, stream, *tensors):
    """The stream's handle; keeps tensors of another stream from being reused
    under this call. The library launches on the current device, and the
    default stream's handle is the same on every device."""
    if _device() != ctx._index:
        raise ValueError(f"the current device is {_device()}, the context's "
                         f"{ctx._index} (torch.cuda.set_device)")
    if stream is None:
        return _raw_stream(ctx._index)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


def _score(score):
    if score not in SCORES:
        raise ValueError(f"score must be one of {list(SCORES)}, got {score!r}")
    return SCORES[score]


def _choice(ctx, T, ids, weights, stream):
    """ids and weights of T tokens, made if not given: (ids, weights)."""
    if ids is None or weights is None:
        make = _maker(ctx, stream)
    if ids is None:
        ids = make((T, ctx.k), torch.int32)
    else:
        _flat(ids, "ids", torch.int32, ctx.device, T * ctx.k)
    if weights is None:
        weights = make((T, ctx.k), torch.float32)
    else:
        _flat(weights, "weights", torch.float32, ctx.device, T * ctx.k)
    return ids, weights


def ue_gate(ctx: Context, logits, bias=None, score="softmax", renorm=True,
            scale=1.0, ids=None, weights=None, stream=None):
    """Expert choice from router logits [T, E] (fp32 or bf16, rows may be
    apart): ids int32 [T, k], best first, and weights fp32 [T, k]. ``ids`` is
    a layer's routing for :func:`ue_load` and :func:`ue_rebalance`."""
    T, _, ld = _rows(logits, "logits", ctx.device, _FLOATS, ctx.E)
    b = None if bias is None else _flat(bias, "bias", torch.float32,
                                        ctx.device, ctx.E)
    ids, weights = _choice(ctx, T, ids, weights, stream)
    rc = library().ue_gate(ctx._h, logits.data_ptr(), _TYPES[logits.dtype],
                           ld, T, _score(score), bool(renorm), scale, b,
                           ids.data_ptr(), weights.data_ptr(),
                           _on(ctx, stream, logits, bias, ids, weights))
    if rc:
        ctx._check(rc, "ue_gate")
    return ids, weights


def ue_gate_backward(ctx: Context, logits, ids, dweights, score="softmax",
                     renorm=True, scale=1.0, dlogits=None, stream=None):
    """Gradient of the logits [T, E] (their type) from the gradient of
    :func:`ue_gate`'s weights, at the same choice and settings."""
    dev = ctx.device
    T, _, ld = _rows(logits, "logits", dev, _FLOATS, ctx.E)
    i = _flat(ids, "ids", torch.int32, dev, T * ctx.k)
    g = _flat(dweights, "dweights", torch.float32, dev, T * ctx.k)
    if dlogits is None:
        dlogits = _new((T, ctx.E), logits.dtype, ctx, stream)
    n, _, ldo = _rows(dlogits, "dlogits", dev, (logits.dtype,), ctx.E)
    if n != T:
        raise ValueError(f"dlogits must have {T} rows")
    rc = library().ue_gate_backward(
        ctx._h, logits.data_ptr(), _TYPES[logits.dtype], ld, T, _score(score),
        bool(renorm), scale, i, g, dlogits.data_ptr(), ldo,
        _on(ctx, stream, logits, ids, dweights, dlogits))
    if rc:
        ctx._check(rc, "ue_gate_backward")
    return dlogits


def ue_quantize_rows(ctx: Context, x, q=None, scale=None, stream=None):
    """Rows of x [M, K] (fp32 or bf16) as int8 [M, K] and scales fp32 [M]. The
    int8 rows are 16-byte aligned (a view of rows padded to a multiple of 16,
    the padding zero)."""
    M, K, ldx = _rows(x, "x", ctx.device, _FLOATS)
    if q is None:
        ldq = (K + 15) // 16 * 16
        q = _new((M, ldq), torch.int8, ctx, stream)
        if ldq != K:
            q = q[:, :K]
    else:
        n, _, ldq = _i8_rows(q, "q", ctx.device, K)
        if n != M:
            raise ValueError(f"q must have {M} rows")
    if scale is None:
        scale = _new((M,), torch.float32, ctx, stream)
    else:
        _flat(scale, "scale", torch.float32, ctx.device, M)
    rc = library().ue_quantize_rows(ctx._h, x.data_ptr(), _TYPES[x.dtype], ldx,
                                    M, K, q.data_ptr(), ldq, scale.data_ptr(),
                                    _on(ctx, stream, x, q, scale))
    if rc:
        ctx._check(rc, "ue_quantize_rows")
    return q, scale


def _i8_rows(t, name, device, cols=None):
    """As _rows; the storage must reach the end of the last row's last
    16-byte piece."""
    n, c, ld = _rows(t, name, device, (torch.int8,), cols)
    if c % 16 and n:
        _i8_reach(t, name, (n - 1) * ld, c)
    return n, c, ld


def _i8_reach(t, name, last_row, cols):
    end = t.storage_offset() + last_row + (cols + 15) // 16 * 16
    if end > t.untyped_storage().nbytes():
        raise ValueError(f"{name}: the last row must be readable up to a "
                         "multiple of 16 bytes")


_PRODUCT = struct.Struct("@8P5q9i")          # ue_i8_product
assert _PRODUCT.size <= ctypes.sizeof(ue_i8_product) < _PRODUCT.size + 8


def ue_matmul_i8(ctx: Context, a, a_scale, w, w_scale, offsets=None,
                 expert_of=None, index=None, index_div=1, gated=False,
                 out=None, out_dtype=torch.bfloat16, stream=None):
    """Product of int8 rows a [rows, K] (scales [rows]) with int8 matrices w
    [N, K] or [experts, N, K] (scales [..., N]); see ``ue_matmul_i8`` in ue.h
    for the row groups (``offsets``, ``expert_of``), the row index and the
    gated form (w with 2 N channels). Rows that no group holds are left as
    they are in ``out``."""
    dev = ctx.device
    rows, K, lda = _i8_rows(a, "a", dev)
    sa = _flat(a_scale, "a_scale", torch.float32, dev, rows)
    if not isinstance(w, torch.Tensor) or w.dtype != torch.int8 or \
            w.device != dev:
        raise TypeError(f"w must be an int8 tensor on {dev}")
    shape, strides = w.shape, w.stride()
    if len(shape) == 2:
        shape, strides = (1, *shape), (0, *strides)
    if len(shape) != 3 or shape[0] < 1 or shape[2] != K:
        raise ValueError(f"w must be [N, {K}] or [experts, N, {K}], is "
                         f"{tuple(w.shape)}")
    n_mats, channels, _ = shape
    w_stride, ldw, one = strides
    if K > 1 and one != 1:
        raise ValueError("w must have contiguous rows")
    if channels <= 1:
        ldw = (K + 15) // 16 * 16
    if n_mats == 1:
        w_stride = 0
    if K % 16 and channels:
        _i8_reach(w, "w", (n_mats - 1) * w_stride + (channels - 1) * ldw, K)
    sw = _flat(w_scale, "w_scale", torch.float32, dev, n_mats * channels)
    N = channels
    if gated:
        if channels % 2:
            raise ValueError("gated: w needs as many up as gate channels")
        N //= 2
    groups, po, pe, pi, M = 0, 0, 0, 0, rows
    if offsets is not None:
        groups = offsets.numel() - 1
        if groups < 0:
            raise ValueError("offsets must hold groups + 1 entries")
        po = _flat(offsets, "offsets", torch.int32, dev, groups + 1)
        if expert_of is not None:
            pe = _flat(expert_of, "expert_of", torch.int32, dev, groups)
    elif expert_of is not None:
        raise ValueError("expert_of needs offsets")
    if index is not None:
        M = index.numel()
        pi = _flat(index, "index", torch.int32, dev, M)
    if out is None:
        out = _new((M, N), out_dtype, ctx, stream)
    n, _, ldo = _rows(out, "out", dev, _FLOATS, N)
    if n != M:
        raise ValueError(f"out must have {M} rows")
    p = _PRODUCT.pack(a.data_ptr(), sa, w.data_ptr(), sw, po, pe, pi,
                      out.data_ptr(), lda, ldw, w_stride, channels, ldo, rows,
                      n_mats, groups, index_div, M, N, K, bool(gated),
                      _TYPES[out.dtype])
    rc = library().ue_matmul_i8(ctx._h, p,
                                _on(ctx, stream, a, a_scale, w, w_scale,
                                    offsets, expert_of, index, out))
    if rc:
        ctx._check(rc, "ue_matmul_i8")
    return out


def ue_register_layer(ctx: Context, router, gate_up, down, gate_up_scale=None,
                      down_scale=None, bias=None, score="softmax",
                      renorm=True, scale=1.0):
    """Registers the layer :func:`ue_moe_tokens` runs: router bf16 [E, H],
    gate_up [E, 2 I, H] (gate rows, then up rows) and down [E, H, I], both
    bf16 or both int8 with channel scales [E, 2 I] and [E, H]. The experts'
    matrices may lie apart (strided in their first dimension). The context
    keeps the tensors until the next registration; a graph captured from
    :func:`ue_moe_tokens` needs the caller to keep its layer's."""
    dev = ctx.device
    _need(router, "router", torch.bfloat16, dev)
    if router.dim() != 2 or router.shape[0] != ctx.E:
        raise ValueError(f"router must be [{ctx.E}, H]")
    H = router.shape[1]
    if gate_up.dtype not in (torch.bfloat16, torch.int8) or \
            down.dtype != gate_up.dtype:
        raise TypeError("gate_up and down must both be bf16 or both int8")
    I = down.shape[-1]
    for t, name, shape in ((gate_up, "gate_up", (ctx.E, 2 * I, H)),
                           (down, "down", (ctx.E, H, I))):
        if t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {shape}, is {tuple(t.shape)}")
        if not t[0].is_contiguous():
            raise ValueError(f"{name}'s matrices must be contiguous")
    i8 = gate_up.dtype == torch.int8
    if i8:
        _need(gate_up_scale, "gate_up_scale", torch.float32, dev, ctx.E * 2 * I)
        _need(down_scale, "down_scale", torch.float32, dev, ctx.E * H)
    elif gate_up_scale is not None or down_scale is not None:
        raise ValueError("scales belong to int8 weights")
    if bias is not None:
        _need(bias, "bias", torch.float32, dev, ctx.E)

    def apart(t):
        return t.stride(0) if ctx.E > 1 else t[0].numel()

    layer = ue_layer(_ptr(router), _ptr(bias), _ptr(gate_up), _ptr(down),
                     _ptr(gate_up_scale), _ptr(down_scale), apart(gate_up),
                     apart(down), H, I, I8 if i8 else BF16, _score(score),
                     bool(renorm), scale)
    with torch.cuda.device(dev):
        rc = library().ue_register_layer(ctx._h, ctypes.byref(layer))
    ctx._check(rc, "ue_register_layer")
    # keep the tensors alive while the library holds their pointers
    ctx._layer = (router, gate_up, down, gate_up_scale, down_scale, bias)
    ctx.hidden = H


def ue_moe_tokens(ctx: Context, x, out=None, ids=None, weights=None,
                  stream=None):
    """The registered layer for x bf16 [T, H], T up to 64: returns (out bf16
    [T, H], ids int32 [T, k], weights fp32 [T, k])."""
    T, H, ldx = _rows(x, "x", ctx.device, (torch.bfloat16,), ctx.hidden)
    if out is None:
        out = _new((T, H), torch.bfloat16, ctx, stream)
    n, _, ldo = _rows(out, "out", ctx.device, (torch.bfloat16,), H)
    if n != T:
        raise ValueError(f"out must have {T} rows")
    ids, weights = _choice(ctx, T, ids, weights, stream)
    rc = library().ue_moe_tokens(ctx._h, x.data_ptr(), ldx, T, out.data_ptr(),
                                 ldo, ids.data_ptr(), weights.data_ptr(),
                                 _on(ctx, stream, x, out, ids, weights))
    if rc:
        ctx._check(rc, "ue_moe_tokens")
    return out, ids, weights


# ---- the expert layer's training step --------------------------------------

PACK_BLOCK = 32        # columns of a packed row that share a power of two


def _sequences(ctx, offsets, name="offsets"):
    """(pointer, sequences) of int32 [n_seq + 1] offsets, or of none."""
    if offsets is None:
        return None, 1
    n = offsets.numel() - 1 if isinstance(offsets, torch.Tensor) else -1
    if n < 0:
        raise ValueError(f"{name} must be a tensor of n_seq + 1 entries")
    return _flat(offsets, name, torch.int32, ctx.device, n + 1), n


def ue_balance(ctx: Context, logits, ids, offsets=None, score="softmax",
               counts=None, prob=None, loss=None, workspace=None, stream=None):
    """Balance loss of packed sequences from router logits [T, E] and the
    choice ids int32 [T, k]: (loss fp32 [n_seq], counts int32 [n_seq, E], prob
    fp32 [n_seq, E]). ``offsets`` int32 [n_seq + 1]: where the sequences start
    (None: all tokens are one). ``workspace``: uint8, of at least
    :func:`ue_balance_workspace` bytes."""
    dev = ctx.device
    T, _, ld = _rows(logits, "logits", dev, _FLOATS, ctx.E)
    i = _flat(ids, "ids", torch.int32, dev, T * ctx.k)
    po, n = _sequences(ctx, offsets)
    score = _score(score)
    if loss is None or counts is None or prob is None:
        make = _maker(ctx, stream)
    if loss is None:
        loss = make((n,), torch.float32)
    else:
        _flat(loss, "loss", torch.float32, dev, n)
    if counts is None:
        counts = make((n, ctx.E), torch.int32)
    else:
        _flat(counts, "counts", torch.int32, dev, n * ctx.E)
    if prob is None:
        prob = make((n, ctx.E), torch.float32)
    else:
        _flat(prob, "prob", torch.float32, dev, n * ctx.E)
    lib = library()
    need, ws = lib.ue_balance_workspace(ctx._h, T, n), None
    if need:
        workspace = _workspace(ctx, workspace, need, stream)
        ws = workspace.data_ptr()
    rc = lib.ue_balance(ctx._h, logits.data_ptr(), _TYPES[logits.dtype],
                              ld, T, score, i, po, n, counts.data_ptr(),
                              prob.data_ptr(), loss.data_ptr(), ws,
                              _on(ctx, stream, logits, ids, offsets, counts,
                                  prob, loss, workspace))
    if rc:
        ctx._check(rc, "ue_balance")
    return loss, counts, prob


def ue_balance_workspace(ctx: Context, T: int, n_seq: int = 1) -> int:
    """Bytes of workspace :func:`ue_balance` needs."""
    return int(library().ue_balance_workspace(ctx._h, T, n_seq))


def _workspace(ctx, t, need, stream):
    if t is None:
        return _new((need,), torch.uint8, ctx, stream)
    _need(t, "workspace", torch.uint8, ctx.device)
    if t.numel() < need:
        raise ValueError(f"workspace must hold {need} bytes, has {t.numel()}")
    return t


def ue_balance_backward(ctx: Context, logits, counts, dloss, offsets=None,
                        score="softmax", dlogits=None, accumulate=False,
                        stream=None):
    """Gradient of the logits [T, E] (their type) from that of the losses
    fp32 [n_seq], at the counts of :func:`ue_balance`. With ``accumulate`` it is
    added to ``dlogits`` (that of :func:`ue_gate_backward`, say)."""
    dev = ctx.device
    T, _, ld = _rows(logits, "logits", dev, _FLOATS, ctx.E)
    po, n = _sequences(ctx, offsets)
    c = _flat(counts, "counts", torch.int32, dev, n * ctx.E)
    d = _flat(dloss, "dloss", torch.float32, dev, n)
    if dlogits is None:
        if accumulate:
            raise ValueError("accumulate needs dlogits to add to")
        dlogits, ldo = _new((T, ctx.E), logits.dtype, ctx, stream), ctx.E
    else:
        rows, _, ldo = _rows(dlogits, "dlogits", dev, (logits.dtype,), ctx.E)
        if rows != T:
            raise ValueError(f"dlogits must have {T} rows")
    rc = library().ue_balance_backward(
        ctx._h, logits.data_ptr(), _TYPES[logits.dtype], ld, T, _score(score),
        po, n, c, d, dlogits.data_ptr(), ldo, bool(accumulate),
        _on(ctx, stream, logits, counts, dloss, offsets, dlogits))
    if rc:
        ctx._check(rc, "ue_balance_backward")
    return dlogits


def _packed_new(make, M, columns):
    """Packed rows of whole blocks: (q int8 [M, P], scale uint8 [M, P / 32])."""
    return (make((M, columns), torch.int8),
            make((M, columns // PACK_BLOCK), torch.uint8))


def _packed(ctx, q, scale, columns=None):
    """(rows, columns, ldq, pointer of q, lds, pointer of scale)."""
    if scale is None:
        raise ValueError("packed rows need their scales")
    M, K, ldq = _rows(q, "q", ctx.device, (torch.int8,), columns)
    blocks = (K + PACK_BLOCK - 1) // PACK_BLOCK
    n, _, lds = _rows(scale, "scale", ctx.device, (torch.uint8,), blocks)
    if n != M:
        raise ValueError(f"scale must have {M} rows")
    if M <= 1:
        # (whole blocks apart, as every call wants them)
        ldq = blocks * PACK_BLOCK
    return M, K, ldq, q.data_ptr(), lds, scale.data_ptr()


def _reach(t, name, rows, ld, cols, unit):
    """The storage must hold the last row up to a multiple of `unit` bytes."""
    if rows and cols % unit:
        end = t.storage_offset() + (rows - 1) * ld + (cols + unit - 1) // unit * unit
        if end > t.untyped_storage().nbytes():
            raise ValueError(f"{name}: the last row must reach a multiple of "
                             f"{unit} bytes")


def ue_pack_rows(ctx: Context, x, q=None, scale=None, stream=None):
    """Rows of x [M, K] (fp32 or bf16) in 8 bits with a power of two per row and
    32 columns: (q int8 [M, K], scale uint8 [M, ceil(K / 32)]). q is a view of
    rows padded with zeros to whole blocks."""
    M, K, ldx = _rows(x, "x", ctx.device, _FLOATS)
    whole = (K + PACK_BLOCK - 1) // PACK_BLOCK * PACK_BLOCK
    if (q is None) != (scale is None):
        raise ValueError("q and scale belong together")
    if q is None:
        q, scale = _packed_new(_maker(ctx, stream), M, whole)
        ldq, lds, pq, ps = whole, whole // PACK_BLOCK, q.data_ptr(), scale.data_ptr()
        if whole != K:
            q = q[:, :K]
    else:
        m, _, ldq, pq, lds, ps = _packed(ctx, q, scale, K)
        if m != M:
            raise ValueError(f"q must have {M} rows")
        _reach(q, "q", M, ldq, K, PACK_BLOCK)
    rc = library().ue_pack_rows(ctx._h, x.data_ptr(), _TYPES[x.dtype], ldx, M,
                                K, pq, ldq, ps, lds,
                                _on(ctx, stream, x, q, scale))
    if rc:
        ctx._check(rc, "ue_pack_rows")
    return q, scale


def ue_unpack_rows(ctx: Context, q, scale, out=None, out_dtype=torch.bfloat16,
                   stream=None):
    """The values [M, K] that packed rows stand for (exact in either type)."""
    M, K, ldq, pq, lds, ps = _packed(ctx, q, scale)
    _reach(q, "q", M, ldq, K, PACK_BLOCK)
    if out is None:
        out = _new((M, K), out_dtype, ctx, stream)
    n, _, ldx = _rows(out, "out", ctx.device, _FLOATS, K)
    if n != M:
        raise ValueError(f"out must have {M} rows")
    rc = library().ue_unpack_rows(ctx._h, pq, ldq, ps, lds, M, K,
                                  out.data_ptr(), _TYPES[out.dtype], ldx,
                                  _on(ctx, stream, q, scale, out))
    if rc:
        ctx._check(rc, "ue_unpack_rows")
    return out


def _out(t, name, ctx, dtype, rows, cols):
    """Distance between the rows of an output [rows, cols] given by the
    caller."""
    n, _, ld = _rows(t, name, ctx.device, (dtype,), cols)
    if n != rows:
        raise ValueError(f"{name} must have {rows} rows")
    return ld


def _half(I):
    """Bytes of gate, and of up, in a packed row of both."""
    return (I + PACK_BLOCK - 1) // PACK_BLOCK * PACK_BLOCK


def ue_gated(ctx: Context, gu, h=None, q=None, scale=None, keep=True,
             stream=None):
    """silu(gate) * up of gu [M, 2 I] (gate, then up): (h [M, I], q int8
    [M, 2 P], scale uint8 [M, P / 16]) with P = I rounded up to 32: gate and up
    as packed rows, gate in q[:, :I], up in q[:, P:P + I]. ``keep=False``: h
    alone is made, q and scale are None."""
    M, two, ldgu = _rows(gu, "gu", ctx.device, _FLOATS)
    if two % 2:
        raise ValueError("gu must hold as many up as gate columns")
    I = two // 2
    make = _maker(ctx, stream) if h is None or (keep and q is None) else None
    if h is None:
        h, ldh = make((M, I), gu.dtype), I
    else:
        ldh = _out(h, "h", ctx, gu.dtype, M, I)
    if (q is None) != (scale is None) or (q is not None and not keep):
        raise ValueError("q and scale belong together, and to keep=True")
    ldq = lds = 0
    pq = ps = None
    if keep and q is None:
        ldq = 2 * _half(I)
        lds = ldq // PACK_BLOCK
        q, scale = _packed_new(make, M, ldq)
        pq, ps = q.data_ptr(), scale.data_ptr()
    elif keep:
        m, _, ldq, pq, lds, ps = _packed(ctx, q, scale, 2 * _half(I))
        if m != M:
            raise ValueError(f"q must have {M} rows")
    rc = library().ue_gated(ctx._h, gu.data_ptr(), _TYPES[gu.dtype], ldgu, M, I,
                            h.data_ptr(), ldh, pq, ldq, ps, lds,
                            _on(ctx, stream, gu, h, q, scale))
    if rc:
        ctx._check(rc, "ue_gated")
    return h, q, scale


def ue_gated_backward(ctx: Context, dh, q, scale, dgu=None, h=None,
                      with_h=True, stream=None):
    """Gradient [M, 2 I] of gate and up from dh [M, I] and what :func:`ue_gated`
    kept, and (``with_h``) silu(gate) * up of the kept values [M, I]:
    (dgu, h)."""
    M, I, lddh = _rows(dh, "dh", ctx.device, _FLOATS)
    m, _, ldq, pq, lds, ps = _packed(ctx, q, scale, 2 * _half(I))
    if m != M:
        raise ValueError(f"q must have {M} rows")
    make = _maker(ctx, stream) if dgu is None or (with_h and h is None) else None
    if dgu is None:
        dgu, lddgu = make((M, 2 * I), dh.dtype), 2 * I
    else:
        lddgu = _out(dgu, "dgu", ctx, dh.dtype, M, 2 * I)
    ldh = I
    if h is not None:
        ldh = _out(h, "h", ctx, dh.dtype, M, I)
    elif with_h:
        h = make((M, I), dh.dtype)
    rc = library().ue_gated_backward(
        ctx._h, pq, ldq, ps, lds, dh.data_ptr(), _TYPES[dh.dtype], lddh, M, I,
        dgu.data_ptr(), lddgu, None if h is None else h.data_ptr(), ldh,
        _on(ctx, stream, q, scale, dh, dgu, h))
    if rc:
        ctx._check(rc, "ue_gated_backward")
    return dgu, h


_WGRAD = struct.Struct("@7P5q7i")            # ue_weight_grad_product
assert _WGRAD.size <= ctypes.sizeof(ue_weight_grad_product) < _WGRAD.size + 8


def ue_weight_grad(ctx: Context, dy, x, x_scale=None, offsets=None, index=None,
                   index_div=1, out=None, accumulate=False, workspace=None,
                   stream=None):
    """Gradients fp32 [groups, N, K] of the matrices of row groups: the sums over
    each group's rows of dy[m]^T x[row of m], dy bf16 [M, N], x bf16 [rows, K]
    or packed (int8 with ``x_scale``). Groups and rows are those of
    :func:`ue_matmul_i8` (``offsets``, ``index``, ``index_div``). With
    ``accumulate`` the sums are added to ``out``. The matrices of ``out`` may lie
    apart, and so may their rows."""
    dev = ctx.device
    M, N, lddy = _rows(dy, "dy", dev, (torch.bfloat16,))
    if x_scale is None:
        rows, K, ldx = _rows(x, "x", dev, (torch.bfloat16,))
        ps, lds = 0, 0
    else:
        rows, K, ldx, _, lds, ps = _packed(ctx, x, x_scale)
        _reach(x, "x", rows, ldx, K, 16)
    groups, po, pi = 1, 0, 0
    if offsets is not None:
        groups = offsets.numel() - 1
        if groups < 0:
            raise ValueError("offsets must hold groups + 1 entries")
        po = _flat(offsets, "offsets", torch.int32, dev, groups + 1)
    if index is not None:
        if index.numel() != M:
            raise ValueError(f"index must hold {M} rows")
        pi = _flat(index, "index", torch.int32, dev, M)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out to add to")
        out = _new((groups, N, K), torch.float32, ctx, stream)
    elif not isinstance(out, torch.Tensor) or out.dtype != torch.float32:
        raise TypeError("out must be an fp32 tensor")
    elif out.device != dev or tuple(out.shape) != (groups, N, K):
        raise ValueError(f"out must be [{groups}, {N}, {K}] on {dev}, is "
                         f"{tuple(out.shape)} on {out.device}")
    out_stride, ldo, one = out.stride()
    if K > 1 and one != 1:
        raise ValueError("out must have contiguous rows")
    if N <= 1:
        ldo = (K + 3) // 4 * 4

    def product(ws):
        return _WGRAD.pack(dy.data_ptr(), x.data_ptr(), ps, po, pi,
                           out.data_ptr(), ws, lddy, ldx, lds, ldo, out_stride,
                           rows, groups, index_div, M, N, K, bool(accumulate))
    p = product(0)
    need = library().ue_weight_grad_workspace(ctx._h, p)
    if need:
        workspace = _workspace(ctx, workspace, need, stream)
        p = product(workspace.data_ptr())
    rc = library().ue_weight_grad(ctx._h, p,
                                  _on(ctx, stream, dy, x, x_scale, offsets,
                                      index, out, workspace))
    if rc:
        ctx._check(rc, "ue_weight_grad")
    return out


def _assigned(ctx, inv_perm, weights):
    """(tokens, pointers) of inv_perm int32 [T, k] and weights fp32 [T, k]."""
    if not isinstance(inv_perm, torch.Tensor) or inv_perm.numel() % ctx.k:
        raise ValueError(f"inv_perm must be an int32 tensor [T, {ctx.k}]")
    T = inv_perm.numel() // ctx.k
    pi = _flat(inv_perm, "inv_perm", torch.int32, ctx.device, T * ctx.k)
    pw = None if weights is None else _flat(weights, "weights", torch.float32,
                                            ctx.device, T * ctx.k)
    return T, pi, pw


def ue_combine(ctx: Context, y, inv_perm, weights=None, add=None, out=None,
               stream=None):
    """out[t] = add[t] + sum_j weights[t, j] y[inv_perm[t, j]]: rows of y [rows,
    H] (fp32 or bf16, dispatch order) back to their tokens. Entries of inv_perm
    outside y's rows add nothing; without weights they are 1 (the gradient of
    :func:`ue_gather_rows`)."""
    dev = ctx.device
    rows, H, ldy = _rows(y, "y", dev, _FLOATS)
    T, pi, pw = _assigned(ctx, inv_perm, weights)
    pa, lda = None, 0
    if add is not None:
        lda = _out(add, "add", ctx, y.dtype, T, H)
        pa = add.data_ptr()
    if out is None:
        out, ldo = _new((T, H), y.dtype, ctx, stream), H
    else:
        ldo = _out(out, "out", ctx, y.dtype, T, H)
    rc = library().ue_combine(ctx._h, y.data_ptr(), _TYPES[y.dtype], ldy, rows,
                              pi, pw, pa, lda, T, H, out.data_ptr(), ldo,
                              _on(ctx, stream, y, inv_perm, weights, add, out))
    if rc:
        ctx._check(rc, "ue_combine")
    return out


def ue_combine_backward(ctx: Context, dout, inv_perm, weights=None, y=None,
                        dy=None, dweights=None, with_dy=True, stream=None):
    """Gradients of :func:`ue_combine` from dout [T, H]: (dy, dweights). dy is
    as y (or, without y, [T * k, H]); its rows that inv_perm does not name are
    zeros, and left as they are in a ``dy`` given by the caller. dweights fp32
    [T, k] needs y and is None without it."""
    dev = ctx.device
    T, H, lddo = _rows(dout, "dout", dev, _FLOATS)
    n, pi, pw = _assigned(ctx, inv_perm, weights)
    if n != T:
        raise ValueError(f"inv_perm must be [{T}, {ctx.k}]")
    if y is None and dweights is not None:
        raise ValueError("dweights needs y")
    rows, ldy, py = T * ctx.k, 0, None
    if (y is not None and dweights is None) or (dy is None and with_dy):
        make = _maker(ctx, stream)
    if y is not None:
        rows, _, ldy = _rows(y, "y", dev, (dout.dtype,), H)
        py = y.data_ptr()
        if dweights is None:
            dweights = make((T, ctx.k), torch.float32)
        else:
            _flat(dweights, "dweights", torch.float32, dev, T * ctx.k)
    lib, lddy = library(), H
    call, ws, workspace = lib.ue_combine_backward, (), None
    if dy is not None:
        n, _, lddy = _rows(dy, "dy", dev, (dout.dtype,), H)
        if y is None:
            rows = n
        elif n != rows:
            raise ValueError(f"dy must have {rows} rows")
    elif with_dy:
        dy = make((rows, H), dout.dtype)
        call, ws = lib.ue_combine_backward_all, (None,)
        need = lib.ue_combine_backward_workspace(ctx._h, T, rows)
        if need:
            workspace = make((need,), torch.uint8)
            ws = (workspace.data_ptr(),)
    rc = call(
        ctx._h, dout.data_ptr(), _TYPES[dout.dtype], lddo, pi, pw, py, ldy,
        rows, T, H, None if dy is None else dy.data_ptr(), lddy,
        None if dweights is None else dweights.data_ptr(), *ws,
        _on(ctx, stream, dout, inv_perm, weights, y, dy, dweights, workspace))
    if rc:
        ctx._check(rc, "ue_combine_backward")
    return dy, dweights
