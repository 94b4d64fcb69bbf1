"""ctypes binding of libgradcomp: the C-ABI calls under the same names.

Argument marshalling only: torch supplies device memory and the current HIP
stream; every step of the computation runs in the library's HIP kernels.
There is no fallback: a missing library raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np
import torch

GC_OK, GC_EINVAL, GC_ECAPACITY, GC_ERANGE, GC_EHIP, GC_ENOTSUP = 0, -1, -2, -3, -4, -5
GC_OP_DGC, GC_OP_ADACOMP, GC_OP_PACK, GC_OP_DECODE, GC_OP_UNPACK = 1, 2, 3, 4, 5
GC_KIND_DGC, GC_KIND_ADACOMP = 1, 2
GC_SUM, GC_AVG = 0, 1
GC_MOMENTUM_VANILLA, GC_MOMENTUM_NESTEROV = 0, 1
GC_SELECT_EXACT, GC_SELECT_SAMPLED = 0, 1
GC_ADACOMP_RULE_RESIDUAL, GC_ADACOMP_RULE_GRADIENT = 0, 1
GC_MAX_BIN_LEN = 4096
GC_MAX_MESSAGES = 64
GC_MAX_SEGMENT_LEN = 0xFFFC0000
GC_MAX_REPLICAS = 16
GC_F32, GC_BF16, GC_F16 = 0, 1, 2
GC_TOKENS_I32, GC_TOKENS_I64 = 0, 1
GC_MUON_SCALE_NONE, GC_MUON_SCALE_SHAPE, GC_MUON_SCALE_RMS = 0, 1, 2
GC_MAX_MATRIX_DIM = 1 << 20
GC_MAX_ORTH_STEPS = 16
GC_ACT_NONE, GC_ACT_RELU, GC_ACT_GELU, GC_ACT_GELU_TANH, GC_ACT_SILU = 0, 1, 2, 3, 4
GC_MAX_VOCAB = 1 << 20
GC_MAX_TOP_LOGITS = 1024
GC_DISTILL_TOP, GC_DISTILL_REST = 0, 1

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgradcomp.so")


class GCError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"libgradcomp status {status}: {msg}")
        self.status = status


class gc_segment(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_uint64), ("length", ctypes.c_uint32),
                ("bin_len", ctypes.c_uint32), ("k", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class gc_sparse(ctypes.Structure):
    _fields_ = [("idx", ctypes.c_void_p), ("val", ctypes.c_void_p),
                ("seg_off", ctypes.c_void_p), ("seg_scale", ctypes.c_void_p),
                ("cap", ctypes.c_uint64)]


class gc_dgc_options(ctypes.Structure):
    _fields_ = [("momentum", ctypes.c_float), ("thr_G", ctypes.c_float),
                ("num_nodes", ctypes.c_int), ("momentum_kind", ctypes.c_int),
                ("select", ctypes.c_int), ("sample_period", ctypes.c_uint32),
                ("over", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
                ("density_num", ctypes.c_uint32), ("density_den", ctypes.c_uint32)]


class gc_adacomp_options(ctypes.Structure):
    _fields_ = [("scale_factor", ctypes.c_float), ("rule", ctypes.c_int),
                ("reserved", ctypes.c_uint32 * 2)]


class gc_orth_options(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int), ("eps", ctypes.c_float),
                ("coef", (ctypes.c_float * 3) * GC_MAX_ORTH_STEPS), ("reserved", ctypes.c_uint32 * 2)]


class gc_muon_options(ctypes.Structure):
    _fields_ = [("orth", gc_orth_options), ("momentum", ctypes.c_float), ("lr", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("momentum_kind", ctypes.c_int), ("scale", ctypes.c_int),
                ("reserved", ctypes.c_uint32)]


class gc_linear(ctypes.Structure):
    _fields_ = [("seg", ctypes.c_int), ("rows", ctypes.c_uint32), ("bias_seg", ctypes.c_int), ("type", ctypes.c_int),
                ("reserved", ctypes.c_uint32 * 2)]


class gc_distill_options(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("kd_weight", ctypes.c_float), ("ce_weight", ctypes.c_float),
                ("grad_scale", ctypes.c_float), ("mode", ctypes.c_int), ("reserved", ctypes.c_uint32 * 3)]


_lib = None

# every symbol the header declares, with (restype, argtypes)
_P = ctypes.c_void_p
_SIGS = {
    "gc_last_error": (ctypes.c_char_p, []),
    "gc_version": (ctypes.c_char_p, []),
    "gc_plan_create": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_uint64, _P]),
    "gc_plan_destroy": (None, [_P]),
    "gc_plan_num_segments": (ctypes.c_int, [_P]),
    "gc_plan_num_elements": (ctypes.c_uint64, [_P]),
    "gc_plan_total_k": (ctypes.c_uint64, [_P]),
    "gc_plan_total_bins": (ctypes.c_uint64, [_P]),
    "gc_topk_count": (ctypes.c_uint32, [ctypes.c_uint32]),
    "gc_plan_workspace_bytes": (ctypes.c_size_t, [_P, ctypes.c_int]),
    "gc_adacomp_compress": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_size_t, ctypes.c_float, _P, _P,
                                           ctypes.c_size_t, _P]),
    "gc_dgc_pack_bound": (ctypes.c_uint64, [_P, _P]),
    "gc_adacomp_compress_ex": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_size_t, _P, _P, _P,
                                              ctypes.c_size_t, _P]),
    "gc_adacomp_state_bytes": (ctypes.c_size_t, [_P]),
    "gc_adacomp_message_cap": (ctypes.c_uint64, [_P]),
    "gc_plan_upload": (ctypes.c_int, [_P]),
    "gc_adacomp_residual": (ctypes.c_int, [_P, _P, _P, ctypes.c_size_t, _P, _P]),
    "gc_dgc_step": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_float, ctypes.c_float, ctypes.c_int,
                                   _P, _P, ctypes.c_size_t, _P]),
    "gc_dgc_message_cap": (ctypes.c_uint64, [_P, _P]),
    "gc_dgc_step_ex": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "gc_pack_bound": (ctypes.c_uint64, [_P, ctypes.c_int]),
    "gc_pack": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, ctypes.c_uint64, _P, _P, ctypes.c_size_t, _P]),
    "gc_unpack": (ctypes.c_int, [_P, ctypes.c_int, _P, ctypes.c_uint64, _P, _P, _P, ctypes.c_size_t, _P]),
    "gc_decompress_accumulate": (ctypes.c_int, [_P, _P, ctypes.c_int, _P, ctypes.c_int, ctypes.c_int,
                                                _P, ctypes.c_size_t, _P]),
    "gc_decompress_noalloc_max_chunks": (ctypes.c_uint64, [ctypes.c_int]),
    "gc_decompress_accumulate_noalloc": (ctypes.c_int, [_P, _P, ctypes.c_int, _P, ctypes.c_int, ctypes.c_int,
                                                        _P]),
    "gc_dcd_compress": (ctypes.c_int, [_P, _P, _P, ctypes.c_uint64, ctypes.c_int, ctypes.c_uint32,
                                       ctypes.c_uint64, ctypes.c_uint64, _P, _P, _P]),
    "gc_dcd_decode": (ctypes.c_int, [_P, _P, ctypes.c_uint64, ctypes.c_int, ctypes.c_uint32, _P, _P]),
    "gc_dcd_mix": (ctypes.c_int, [_P, _P, ctypes.c_int, _P, ctypes.c_float, _P, ctypes.c_uint64, _P]),
    "gc_ecd_compress": (ctypes.c_int, [_P, _P, ctypes.c_uint64, ctypes.c_uint64, ctypes.c_int,
                                       ctypes.c_uint32, ctypes.c_uint64, _P, _P, _P]),
    "gc_ecd_update": (ctypes.c_int, [_P, _P, ctypes.c_uint64, ctypes.c_int, ctypes.c_uint32,
                                     ctypes.c_uint64, _P, _P]),
    "gc_slimdp_mask_words": (ctypes.c_uint64, [_P]),
    "gc_slimdp_core": (ctypes.c_int, [_P, _P, _P, ctypes.c_float, _P, _P, _P, ctypes.c_size_t, _P]),
    "gc_slimdp_explore": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_uint64, ctypes.c_uint64, _P, _P,
                                         ctypes.c_size_t, _P]),
    "gc_slimdp_core_values": (ctypes.c_int, [_P, _P, _P, _P, _P]),
    "gc_embed_lookup": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_uint32, _P, _P, ctypes.c_int, ctypes.c_uint64,
                                       ctypes.c_float, _P, ctypes.c_int, ctypes.c_uint64, _P]),
    "gc_embed_workspace_bytes": (ctypes.c_size_t, [_P, ctypes.c_int, ctypes.c_uint32, ctypes.c_uint64]),
    "gc_embed_grad": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_uint32, _P, ctypes.c_int, ctypes.c_uint64, _P,
                                     ctypes.c_int, ctypes.c_uint64, ctypes.c_float, _P, ctypes.c_int, _P,
                                     ctypes.c_size_t, _P]),
    "gc_embed_message_cap": (ctypes.c_uint64, [_P, ctypes.c_int, ctypes.c_uint32, ctypes.c_uint64]),
    "gc_embed_message": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_uint32, _P, ctypes.c_int, ctypes.c_uint64, _P,
                                        ctypes.c_int, ctypes.c_uint64, ctypes.c_float, _P, _P, ctypes.c_size_t, _P]),
    "gc_matrix_plan_create": (ctypes.c_int, [_P, _P, _P]),
    "gc_matrix_plan_destroy": (None, [_P]),
    "gc_matrix_plan_upload": (ctypes.c_int, [_P]),
    "gc_matrix_plan_workspace_bytes": (ctypes.c_size_t, [_P]),
    "gc_orthogonalize": (ctypes.c_int, [_P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "gc_muon_step": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "gc_linear_workspace_bytes": (ctypes.c_size_t, [_P, _P, ctypes.c_uint64]),
    "gc_linear_forward": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_uint64, ctypes.c_uint64, ctypes.c_int, _P,
                                         ctypes.c_uint64, _P, ctypes.c_uint64, _P, ctypes.c_uint64, _P, ctypes.c_size_t,
                                         _P]),
    "gc_act_grad": (ctypes.c_int, [_P, ctypes.c_uint64, _P, ctypes.c_uint64, ctypes.c_int, ctypes.c_int, ctypes.c_uint64,
                                   ctypes.c_uint64, _P, ctypes.c_uint64, _P]),
    "gc_linear_grad_input": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_uint64, ctypes.c_uint64, _P, ctypes.c_uint64,
                                            ctypes.c_int, _P, ctypes.c_uint64, _P, ctypes.c_uint64, _P, ctypes.c_uint64,
                                            _P, ctypes.c_size_t, _P]),
    "gc_linear_grad_weight": (ctypes.c_int, [_P, _P, _P, ctypes.c_uint64, _P, ctypes.c_uint64, ctypes.c_uint64, _P,
                                             ctypes.c_int, _P, ctypes.c_size_t, _P]),
    "gc_top_logits": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_uint64, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_uint32,
                                     ctypes.c_float, _P, _P, _P, _P]),
    "gc_distill_loss": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_uint64, ctypes.c_uint64, ctypes.c_uint32, _P,
                                       ctypes.c_int, ctypes.c_uint64, _P, ctypes.c_int, ctypes.c_uint64, ctypes.c_uint32,
                                       _P, _P, _P, _P, _P, _P, ctypes.c_uint64, _P]),
    "gc_timing_enable": (ctypes.c_int, [ctypes.c_char_p]),
    "gc_timing_take": (ctypes.c_int, [ctypes.c_char_p, _P, _P]),
    "gc_stream_probe": (ctypes.c_int, [_P, _P, _P, _P, _P, ctypes.c_uint64, _P]),
}

KERNELS = ("dgc_norm", "dgc_prep", "dgc_prepare", "dgc_sample", "dgc_bound", "dgc_ssample", "dgc_squant", "dgc_update", "dgc_collect",
           "dgc_select", "dgc_stage", "dgc_refine", "dgc_sbase", "dgc_count", "dgc_scan", "dgc_emit", "ada_max", "ada_binsum", "ada_scale", "ada_offsets", "ada_apply",
           "ada_fold", "ada_emit", "ada_residual",
           "pack_plan", "pack_write", "pack_relayout", "pack_rewrite", "pack_main", "pack_fix", "unpack_layout",
           "unpack_write", "decode_index", "decode", "dcd",
           "dcd_decode", "dcd_mix", "ecd_compress", "ecd_update", "slimdp_values", "stream_probe",
           "embed_lookup", "embed_rank", "embed_merge", "embed_heads", "embed_rows", "embed_sum", "embed_join",
           "embed_small", "embed_empty", "orth_norm", "orth_scale", "orth_split", "orth_gram", "orth_poly", "orth_pair", "orth_apply", "orth_join",
           "orth_slab", "orth_small", "linear_product", "linear_few", "linear_join", "act_grad", "top_logits", "distill")


def gc_timing_enable(kernels) -> None:
    """Bracket launches of the named kernels with HIP events ("*" = all,
    None or "" = off)."""
    if kernels is None:
        arg = None
    elif isinstance(kernels, str):
        arg = kernels.encode()
    else:
        arg = ",".join(kernels).encode()
    _check(load().gc_timing_enable(arg))


def gc_stream_probe(a, b, c, d, e) -> None:
    """The streaming reference: d = a + b, e = c + d over a.numel() fp32
    elements (three reads, two writes per element)."""
    n = a.numel()
    _check(load().gc_stream_probe(_f32(a, n, "a"), _f32(b, n, "b"), _f32(c, n, "c"), _f32(d, n, "d"),
                                  _f32(e, n, "e"), n, _stream(d)))


def gc_timing_take(kernel: str):
    """(total milliseconds, launches) recorded for a kernel since the last take."""
    ms = ctypes.c_double()
    n = ctypes.c_uint64()
    _check(load().gc_timing_take(kernel.encode(), ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value


def load():
    """Load libgradcomp.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def exported_symbols():
    return list(_SIGS)


def _check(status: int):
    if status != GC_OK:
        raise GCError(status, load().gc_last_error().decode())


def gc_version() -> str:
    return load().gc_version().decode()


def gc_last_error() -> str:
    return load().gc_last_error().decode()


def gc_topk_count(n: int) -> int:
    return int(load().gc_topk_count(int(n)))


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


_Tensor = torch.Tensor


# The C ABI trusts the sizes it is given; these checks make every pointer the
# binding passes down a contiguous CUDA tensor of the right type holding at
# least the elements the call may touch.
def _dev(t, dtype, n: int, name: str):
    if not isinstance(t, _Tensor) or t.dtype is not dtype or not t.is_cuda or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name}: need a contiguous CUDA {str(dtype).replace('torch.', '')} tensor "
                         f"of >= {n} elements")
    return t.data_ptr()


def _f32(t: torch.Tensor, n: int, name: str):
    return _dev(t, torch.float32, n, name)


def _ws(ws: torch.Tensor, name: str = "ws"):
    """A workspace: uint8, so that its element count is its byte count."""
    return _dev(ws, torch.uint8, 1, name), ws.numel()


def _state(state):
    return ctypes.c_void_p(0) if state is None else _dev(state, torch.uint8, 1, "state")


# ---------------------------------------------------------------- plans
class Plan:
    """A validated segment table (gc_plan)."""

    def __init__(self, table, n_total: int | None = None):
        t = np.asarray(table, dtype=np.int64).reshape(-1, 4)
        self.table = t
        self.lengths = t[:, 1].tolist()
        self.n_total = int(n_total if n_total is not None else (t[-1, 0] + t[-1, 1] if len(t) else 0))
        arr = (gc_segment * max(len(t), 1))()
        for i, (o, n, lt, k) in enumerate(t):
            arr[i] = gc_segment(int(o), int(n), int(lt), int(k), 0)
        h = ctypes.c_void_p()
        _check(load().gc_plan_create(arr, len(t), self.n_total, ctypes.byref(h)))
        self.handle = h
        self.nseg = len(t)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib is not None:
            _lib.gc_plan_destroy(h)
            self.handle = None

    @property
    def total_k(self) -> int:
        return int(load().gc_plan_total_k(self.handle))

    @property
    def total_bins(self) -> int:
        return int(load().gc_plan_total_bins(self.handle))

    def upload(self) -> None:
        """Put the plan's tables on the current device (gc_plan_upload)."""
        _check(load().gc_plan_upload(self.handle))

    def workspace_bytes(self, op: int) -> int:
        return int(load().gc_plan_workspace_bytes(self.handle, op))

    def workspace(self, op: int, device="cuda") -> torch.Tensor:
        return torch.empty(max(self.workspace_bytes(op), 1), dtype=torch.uint8, device=device)

    def pack_bound(self, kind: int) -> int:
        return int(load().gc_pack_bound(self.handle, kind))

    @property
    def adacomp_state_bytes(self) -> int:
        return int(load().gc_adacomp_state_bytes(self.handle))

    def adacomp_state(self, device="cuda") -> torch.Tensor:
        """A zero-filled deferred-residual state for one learner (torch
        allocations are 256-byte aligned)."""
        return torch.zeros(max(self.adacomp_state_bytes, 1), dtype=torch.uint8, device=device)


def gc_plan_create(table, n_total=None) -> Plan:
    return Plan(table, n_total)


def gc_plan_workspace_bytes(plan: Plan, op: int) -> int:
    return plan.workspace_bytes(op)


def gc_pack_bound(plan: Plan, kind: int) -> int:
    return plan.pack_bound(kind)


@dataclass
class Sparse:
    """A message: device tensors idx (int32 holding u32), val, seg_off, seg_scale."""
    idx: torch.Tensor
    val: torch.Tensor
    seg_off: torch.Tensor
    seg_scale: torch.Tensor
    cap: int

    @staticmethod
    def empty(plan: Plan, cap: int, device="cuda") -> "Sparse":
        return Sparse(torch.zeros(max(cap, 1), dtype=torch.int32, device=device),
                      torch.zeros(max(cap, 1), dtype=torch.float32, device=device),
                      torch.zeros(plan.nseg + 1, dtype=torch.int32, device=device),
                      torch.zeros(max(plan.nseg, 1), dtype=torch.float32, device=device), cap)

    def struct(self) -> gc_sparse:
        return gc_sparse(self.idx.data_ptr(), self.val.data_ptr(), self.seg_off.data_ptr(),
                         self.seg_scale.data_ptr(), self.cap)

    def checked(self, plan: "Plan", name: str = "message") -> gc_sparse:
        """The struct, after checking that the tensors hold cap entries and
        the plan's per-segment arrays."""
        i32, f32, nseg = torch.int32, torch.float32, plan.nseg
        return gc_sparse(_dev(self.idx, i32, self.cap, name + ".idx"), _dev(self.val, f32, self.cap, name + ".val"),
                         _dev(self.seg_off, i32, nseg + 1, name + ".seg_off"),
                         _dev(self.seg_scale, f32, nseg or 1, name + ".seg_scale"), self.cap)

    def count(self) -> int:
        return int(self.seg_off[-1].item())

    def host(self):
        """(idx u32, val f32, seg_off u32, seg_scale f32) as NumPy arrays."""
        n = self.count()
        return (self.idx[:n].cpu().numpy().view(np.uint32), self.val[:n].cpu().numpy(),
                self.seg_off.cpu().numpy().view(np.uint32), self.seg_scale.cpu().numpy())


# -------------------------------------------------------------- hot calls
def gc_adacomp_compress(plan: Plan, dW, R, scale_factor: float, out: Sparse, ws: torch.Tensor,
                        state: torch.Tensor | None = None, rule: int | None = None):
    """state None: R is the exact residual.  state (Plan.adacomp_state()):
    deferred mode, the residual is (R, state).  rule None:
    gc_adacomp_compress (the default reading); else gc_adacomp_compress_ex
    with that GC_ADACOMP_RULE_*."""
    n = plan.n_total
    msg = out.checked(plan, "out")
    args = (plan.handle, _f32(dW, n, "dW"), _f32(R, n, "R"), _state(state),
            state.numel() if state is not None else 0)
    if rule is None:
        _check(load().gc_adacomp_compress(*args, float(scale_factor), ctypes.byref(msg), *_ws(ws), _stream(R)))
    else:
        opt = gc_adacomp_options(float(scale_factor), int(rule))
        _check(load().gc_adacomp_compress_ex(*args, ctypes.byref(opt), ctypes.byref(msg), *_ws(ws), _stream(R)))


def gc_adacomp_message_cap(plan: Plan) -> int:
    """Slots an AdaComp message needs: the sum of the segment lengths."""
    return int(load().gc_adacomp_message_cap(plan.handle))


def gc_adacomp_state_bytes(plan: Plan) -> int:
    return plan.adacomp_state_bytes


def gc_adacomp_residual(plan: Plan, R, state: torch.Tensor | None, R_out):
    n = plan.n_total
    _check(load().gc_adacomp_residual(plan.handle, _f32(R, n, "R"), _state(state),
                                      state.numel() if state is not None else 0,
                                      _f32(R_out, n, "R_out"), _stream(R_out)))


def gc_dgc_step(plan: Plan, G, U, V, momentum: float, thr_G: float, num_nodes: int, out: Sparse,
                ws: torch.Tensor):
    n = plan.n_total
    msg = out.checked(plan, "out")
    _check(load().gc_dgc_step(plan.handle, _f32(G, n, "G"), _f32(U, n, "U"), _f32(V, n, "V"),
                              float(momentum), float(thr_G), int(num_nodes), ctypes.byref(msg),
                              *_ws(ws), _stream(V)))


def dgc_options(momentum: float, thr_G: float = 0.0, num_nodes: int = 1, nesterov: bool = False,
                sampled: bool = False, sample_period: int = 100, over: int = 2,
                density: tuple[int, int] | None = None) -> gc_dgc_options:
    """density=(num, den): this call keeps ceil(n_s num / den) entries per
    segment instead of the plan's k (warm-up)."""
    num, den = density if density is not None else (0, 0)
    return gc_dgc_options(float(momentum), float(thr_G), int(num_nodes),
                          GC_MOMENTUM_NESTEROV if nesterov else GC_MOMENTUM_VANILLA,
                          GC_SELECT_SAMPLED if sampled else GC_SELECT_EXACT,
                          int(sample_period), int(over), 0, int(num), int(den))


def gc_dgc_message_cap(plan: Plan, opt: gc_dgc_options) -> int:
    return int(load().gc_dgc_message_cap(plan.handle, ctypes.byref(opt)))


def gc_dgc_pack_bound(plan: Plan, opt: gc_dgc_options | None) -> int:
    return int(load().gc_dgc_pack_bound(plan.handle, ctypes.byref(opt) if opt is not None else None))


def gc_dgc_step_ex(plan: Plan, G, U, V, opt: gc_dgc_options, out: Sparse, ws: torch.Tensor):
    n = plan.n_total
    msg = out.checked(plan, "out")
    _check(load().gc_dgc_step_ex(plan.handle, _f32(G, n, "G"), _f32(U, n, "U"), _f32(V, n, "V"),
                                 ctypes.byref(opt), ctypes.byref(msg), *_ws(ws), _stream(V)))


def gc_pack(plan: Plan, kind: int, msg: Sparse, out: torch.Tensor, out_bytes: torch.Tensor,
            ws: torch.Tensor):
    if out.dtype != torch.uint8 or out_bytes.dtype != torch.int64:
        raise ValueError("gc_pack: out must be uint8 and out_bytes int64 (holding u64)")
    m = msg.checked(plan, "msg")
    _check(load().gc_pack(plan.handle, int(kind), ctypes.byref(m), _dev(out, torch.uint8, 1, "out"), out.numel(),
                          _dev(out_bytes, torch.int64, 1, "out_bytes"), *_ws(ws), _stream(out)))


def gc_unpack(plan: Plan, kind: int, data: torch.Tensor, nbytes: int, out: Sparse, status: torch.Tensor,
              ws: torch.Tensor):
    """data: uint8 device tensor holding the stream's nbytes bytes; status:
    an int32 device tensor (holding u32) that receives the stream's status."""
    if data.dtype != torch.uint8 or data.numel() < nbytes or status.dtype != torch.int32:
        raise ValueError("gc_unpack: data must be uint8 with nbytes bytes, status int32")
    m = out.checked(plan, "out")
    _check(load().gc_unpack(plan.handle, int(kind), _dev(data, torch.uint8, nbytes, "data"), int(nbytes), ctypes.byref(m), _dev(status, torch.int32, 1, "status"),
                            *_ws(ws), _stream(data)))


def gc_decompress_accumulate(plan: Plan, msgs, dense, mode: int, accumulate: bool,
                             ws: torch.Tensor):
    K = len(msgs)
    arr = (gc_sparse * max(K, 1))(*[m.checked(plan, f"msgs[{i}]") for i, m in enumerate(msgs)])
    _check(load().gc_decompress_accumulate(plan.handle, arr, K, _f32(dense, plan.n_total, "dense"),
                                           int(mode), int(bool(accumulate)), *_ws(ws),
                                           _stream(dense)))


def gc_decompress_noalloc_max_chunks(K: int) -> int:
    return int(load().gc_decompress_noalloc_max_chunks(int(K)))


def gc_decompress_accumulate_noalloc(plan: Plan, msgs, dense, mode: int, accumulate: bool):
    """gc_decompress_accumulate with the library's fixed device scratch in
    place of a workspace; the plan must have been uploaded (Plan.upload)."""
    K = len(msgs)
    arr = (gc_sparse * max(K, 1))(*[m.checked(plan, f"msgs[{i}]") for i, m in enumerate(msgs)])
    _check(load().gc_decompress_accumulate_noalloc(plan.handle, arr, K, _f32(dense, plan.n_total, "dense"),
                                                   int(mode), int(bool(accumulate)), _stream(dense)))


def gc_dcd_compress(x, x_half, x_out, bits: int, bucket: int, seed: int, step: int,
                    scales: torch.Tensor, codes: torch.Tensor):
    n = x.numel()
    nb = (n + bucket - 1) // bucket
    if scales.numel() < nb or codes.numel() < (n * bits + 7) // 8 or codes.dtype != torch.uint8:
        raise ValueError("gc_dcd_compress: scales or codes too small")
    _check(load().gc_dcd_compress(_f32(x, n, "x"), _f32(x_half, n, "x_half"), _f32(x_out, n, "x_out"),
                                  n, int(bits), int(bucket), int(seed) & (2 ** 64 - 1),
                                  int(step) & (2 ** 64 - 1), _f32(scales, nb, "scales"), _dev(codes, torch.uint8, (n * bits + 7) // 8, "codes"),
                                  _stream(x_out)))


def _codes_check(n: int, bits: int, bucket: int, scales: torch.Tensor, codes: torch.Tensor, fn: str):
    nb = (n + bucket - 1) // bucket
    if scales.numel() < nb or codes.numel() < (n * bits + 7) // 8 or codes.dtype != torch.uint8:
        raise ValueError(f"{fn}: scales or codes too small")
    return nb


def gc_dcd_decode(scales: torch.Tensor, codes: torch.Tensor, x_hat, bits: int, bucket: int):
    n = x_hat.numel()
    nb = _codes_check(n, bits, bucket, scales, codes, "gc_dcd_decode")
    _check(load().gc_dcd_decode(_f32(scales, nb, "scales"), _dev(codes, torch.uint8, (n * bits + 7) // 8, "codes"), n, int(bits), int(bucket),
                                _f32(x_hat, n, "x_hat"), _stream(x_hat)))


def gc_dcd_mix(replicas, weights, grad, lr: float, x_half):
    n = x_half.numel()
    K = len(replicas)
    reps = (ctypes.c_void_p * max(K, 1))(*[_f32(r, n, "replica") for r in replicas])
    w = (ctypes.c_float * max(K, 1))(*[float(v) for v in weights])
    _check(load().gc_dcd_mix(reps, w, K, _f32(grad, n, "grad"), float(lr), _f32(x_half, n, "x_half"), n,
                             _stream(x_half)))


def gc_ecd_compress(x_prev, x, t: int, bits: int, bucket: int, seed: int, scales: torch.Tensor,
                    codes: torch.Tensor):
    n = x.numel()
    nb = _codes_check(n, bits, bucket, scales, codes, "gc_ecd_compress")
    _check(load().gc_ecd_compress(_f32(x_prev, n, "x_prev"), _f32(x, n, "x"), n, int(t), int(bits),
                                  int(bucket), int(seed) & (2 ** 64 - 1), _f32(scales, nb, "scales"),
                                  _dev(codes, torch.uint8, (n * bits + 7) // 8, "codes"), _stream(x)))


def gc_ecd_update(scales: torch.Tensor, codes: torch.Tensor, x_tilde, t: int, bits: int, bucket: int):
    n = x_tilde.numel()
    nb = _codes_check(n, bits, bucket, scales, codes, "gc_ecd_update")
    _check(load().gc_ecd_update(_f32(scales, nb, "scales"), _dev(codes, torch.uint8, (n * bits + 7) // 8, "codes"), n, int(bits), int(bucket), int(t),
                                _f32(x_tilde, n, "x_tilde"), _stream(x_tilde)))


def gc_slimdp_mask_words(plan: Plan) -> int:
    return int(load().gc_slimdp_mask_words(plan.handle))


def gc_slimdp_core(plan: Plan, w, g, c: float, core: Sparse, core_mask: torch.Tensor, ws: torch.Tensor):
    n = plan.n_total
    if core_mask.dtype != torch.int32 or core_mask.numel() < gc_slimdp_mask_words(plan):
        raise ValueError("gc_slimdp_core: core_mask must be int32 (holding u32) of gc_slimdp_mask_words words")
    msg = core.checked(plan, "core")
    _check(load().gc_slimdp_core(plan.handle, _f32(w, n, "w"), _f32(g, n, "g"), float(c), ctypes.byref(msg),
                                 _dev(core_mask, torch.int32, gc_slimdp_mask_words(plan), "core_mask"), *_ws(ws), _stream(core_mask)))


def gc_slimdp_explore(plan: Plan, core_plan: Plan, delta, core_mask: torch.Tensor, seed: int, step: int,
                      out: Sparse, ws: torch.Tensor):
    n = plan.n_total
    msg = out.checked(plan, "out")
    _check(load().gc_slimdp_explore(plan.handle, core_plan.handle, _f32(delta, n, "delta"), _dev(core_mask, torch.int32, gc_slimdp_mask_words(plan), "core_mask"),
                                    int(seed) & (2 ** 64 - 1), int(step) & (2 ** 64 - 1), ctypes.byref(msg),
                                    *_ws(ws), _stream(delta)))


def gc_slimdp_core_values(core_plan: Plan, core: Sparse, delta, values):
    msg = core.checked(core_plan, "core")
    _check(load().gc_slimdp_core_values(core_plan.handle, ctypes.byref(msg), _f32(delta, core_plan.n_total, "delta"),
                                        _f32(values, core_plan.total_k, "values"), _stream(values)))


# ------------------------------------------------------------- embedding
_FLOAT_TYPES = {torch.float32: GC_F32, torch.bfloat16: GC_BF16, torch.float16: GC_F16}
_TOKEN_TYPES = {torch.int32: GC_TOKENS_I32, torch.int64: GC_TOKENS_I64}


def _row_stride(t, name: str) -> int:
    """The one stride between a batch's rows, which are contiguous in themselves."""
    cols = t.shape[-1]
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    stride, step = None, None
    for size, st in list(zip(t.shape[:-1], t.stride()[:-1]))[::-1]:  # each must continue the one behind it
        if size == 1:
            continue
        if stride is None:
            stride = st
        elif st != step:
            raise ValueError(f"{name}: rows must be one stride apart")
        step = st * size
    stride = cols if stride is None else stride
    if stride < cols:
        raise ValueError(f"{name}: rows must not overlap")
    return stride


def _batch(plan: Plan, seg: int, rows: int, tokens, t, name: str):
    """(t pointer, GC_* type, row stride), (tokens pointer, GC_TOKENS_*, count)
    of a batch (_call checks the devices): tokens contiguous, of any shape; t their shape with the
    columns of segment seg, read as rows x columns, appended."""
    if not 0 <= seg < plan.nseg or rows < 1 or plan.lengths[seg] % rows:
        raise ValueError("seg must be a segment of the plan and rows divide its length")
    if not isinstance(tokens, _Tensor) or not isinstance(t, _Tensor) or not tokens.is_contiguous():
        raise ValueError(f"tokens, {name}: need tensors, tokens contiguous")
    cols, token_type, kind = plan.lengths[seg] // rows, _TOKEN_TYPES.get(tokens.dtype), _FLOAT_TYPES.get(t.dtype)
    if token_type is None:
        raise ValueError("tokens: need int32 or int64")
    if kind is None or t.shape != (*tokens.shape, cols):
        raise ValueError(f"{name}: need an fp32, bf16 or fp16 tensor of shape {(*tokens.shape, cols)}")
    stride = cols if t.is_contiguous() else _row_stride(t, name)
    return (t.data_ptr(), kind, stride), (tokens.data_ptr(), token_type, tokens.numel())


# the raw handle without a Stream object around it (about 1 us less per call),
# and the device without the check that CUDA is initialised, which its tensors show
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(fn: str, tensors, *args):
    """The library's call on the tensors' device, made the current one (the
    library enqueues there), and on that device's current stream."""
    index = tensors[0].get_device()  # -1 for the CPU
    for t in tensors:
        if t.get_device() != index or index < 0:
            raise ValueError("need CUDA tensors on one device")
    if _device() == index:
        status = getattr(_lib or load(), fn)(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = getattr(load(), fn)(*args, _raw_stream(index))
    if status != GC_OK:
        _check(status)


def gc_embed_lookup(plan: Plan, seg: int, rows: int, w, tokens: torch.Tensor, scale: float, y: torch.Tensor):
    """y[...] = scale * w's row tokens[...]; y has the tokens' shape with the
    columns appended, in fp32, bf16 or fp16, its rows one stride apart."""
    batch, toks = _batch(plan, seg, rows, tokens, y, "y")
    wp = _f32(w, plan.n_total, "w")
    _call("gc_embed_lookup", (y, tokens, w), plan.handle, seg, rows, wp, *toks, scale, *batch)


def gc_embed_workspace_bytes(plan: Plan, seg: int, rows: int, n_tokens: int) -> int:
    return int(load().gc_embed_workspace_bytes(plan.handle, int(seg), int(rows), int(n_tokens)))


def gc_embed_grad(plan: Plan, seg: int, rows: int, dy: torch.Tensor, tokens: torch.Tensor, scale: float, g,
                  accumulate: bool, ws: torch.Tensor):
    """The lookup's gradient, written over (accumulate False) or added to
    segment seg of g; dy as gc_embed_lookup's y."""
    batch, toks = _batch(plan, seg, rows, tokens, dy, "dy")
    gp, space = _f32(g, plan.n_total, "g"), _ws(ws)
    _call("gc_embed_grad", (g, dy, tokens, ws), plan.handle, seg, rows, *batch, *toks, scale, gp,
          int(bool(accumulate)), *space)


def gc_embed_message_cap(plan: Plan, seg: int, rows: int, n_tokens: int) -> int:
    return int(load().gc_embed_message_cap(plan.handle, int(seg), int(rows), int(n_tokens)))


def gc_embed_message(plan: Plan, seg: int, rows: int, dy: torch.Tensor, tokens: torch.Tensor, scale: float,
                     out: Sparse, ws: torch.Tensor):
    """The lookup's gradient as a message of the rows that have tokens."""
    batch, toks = _batch(plan, seg, rows, tokens, dy, "dy")
    msg, space = out.checked(plan, "out"), _ws(ws)
    _call("gc_embed_message", (out.val, out.idx, out.seg_off, dy, tokens, ws), plan.handle, seg, rows, *batch, *toks,
          scale, ctypes.byref(msg), *space)


# -------------------------------------------------------- matrix updates
class MatrixPlan:
    """The weight matrices among a plan's segments (gc_matrix_plan): rows[s]
    is segment s's row count, 0 for a segment that is no matrix."""

    def __init__(self, plan: Plan, rows):
        r = np.asarray(rows, dtype=np.int64).reshape(-1)
        if len(r) != plan.nseg or (r < 0).any() or (r > 0xFFFFFFFF).any():
            raise ValueError("rows: need one count >= 0 per segment of the plan")
        self.n_total = plan.n_total
        arr = (ctypes.c_uint32 * len(r))(*[int(v) for v in r])
        h = ctypes.c_void_p()
        _check(load().gc_matrix_plan_create(plan.handle, arr, ctypes.byref(h)))
        self.handle = h

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib is not None:
            _lib.gc_matrix_plan_destroy(h)
            self.handle = None

    def upload(self) -> None:
        """Put the tables on the current device (gc_matrix_plan_upload)."""
        _check(load().gc_matrix_plan_upload(self.handle))

    def workspace_bytes(self) -> int:
        return int(load().gc_matrix_plan_workspace_bytes(self.handle))

    def workspace(self, device="cuda") -> torch.Tensor:
        return torch.empty(self.workspace_bytes(), dtype=torch.uint8, device=device)


def orth_options(steps: int = 5, coef=(3.4445, -4.7750, 2.0315), eps: float = 1e-7) -> gc_orth_options:
    """coef: (a, b, c) for every step, or one such triple per step."""
    each = [tuple(coef)] * steps if np.ndim(coef) == 1 else [tuple(c) for c in coef]
    if len(each) != steps or any(len(c) != 3 for c in each):
        raise ValueError("coef: need (a, b, c), or one triple per step")
    o = gc_orth_options(int(steps), float(eps))
    for k, c in enumerate(each[:GC_MAX_ORTH_STEPS]):
        o.coef[k][:] = [float(v) for v in c]
    return o


def muon_options(momentum: float, lr: float, weight_decay: float = 0.0, nesterov: bool = True,
                 scale: int = GC_MUON_SCALE_SHAPE, steps: int = 5, coef=(3.4445, -4.7750, 2.0315),
                 eps: float = 1e-7) -> gc_muon_options:
    return gc_muon_options(orth_options(steps, coef, eps), float(momentum), float(lr), float(weight_decay),
                           GC_MOMENTUM_NESTEROV if nesterov else GC_MOMENTUM_VANILLA, int(scale), 0)


def gc_orthogonalize(mplan: MatrixPlan, D, O, opt: gc_orth_options, ws: torch.Tensor):
    """Every matrix of D orthogonalised into O (which may be D)."""
    n = mplan.n_total
    args = _f32(D, n, "D"), _f32(O, n, "O"), ctypes.byref(opt), *_ws(ws)
    _call("gc_orthogonalize", (O, D, ws), mplan.handle, *args)


def gc_muon_step(mplan: MatrixPlan, G, U, W, opt: gc_muon_options, ws: torch.Tensor):
    """U <- m U + G, W <- (1 - lr wd) W - lr s orthogonalised(D) on every matrix."""
    n = mplan.n_total
    args = _f32(G, n, "G"), _f32(U, n, "U"), _f32(W, n, "W"), ctypes.byref(opt), *_ws(ws)
    _call("gc_muon_step", (W, G, U, ws), mplan.handle, *args)


# ------------------------------------------------------- layer products
def linear_layer(seg: int, rows: int, dtype=torch.float32, bias_seg: int = -1) -> gc_linear:
    """The layer whose weights are segment seg, read as rows x columns, with
    activations (and the copy of the flat model) in dtype."""
    if dtype not in _FLOAT_TYPES:
        raise ValueError("dtype: need torch.float32, bfloat16 or float16")
    return gc_linear(int(seg), int(rows), int(bias_seg), _FLOAT_TYPES[dtype])


_DTYPES = {v: k for k, v in _FLOAT_TYPES.items()}
_ABSENT = (None, 0)


def _layer_cols(plan: Plan, layer: gc_linear) -> int:
    if not 0 <= layer.seg < plan.nseg or layer.rows < 1 or plan.lengths[layer.seg] % layer.rows:
        raise ValueError("seg must be a segment of the plan and rows divide its length")
    if layer.type not in _DTYPES:
        raise ValueError("type: need GC_F32, GC_BF16 or GC_F16")
    return plan.lengths[layer.seg] // layer.rows


def _acts(t, dtype, shape, name: str):
    """(pointer, row stride) of activations of the given shape, rows one stride apart."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: need a {str(dtype).replace('torch.', '')} tensor of shape {tuple(shape)}")
    return t.data_ptr(), shape[-1] if t.is_contiguous() else _row_stride(t, name)


def gc_linear_workspace_bytes(plan: Plan, layer: gc_linear, n_tokens: int) -> int:
    return int(load().gc_linear_workspace_bytes(plan.handle, ctypes.byref(layer), int(n_tokens)))


def gc_linear_forward(plan: Plan, layer: gc_linear, w, x: torch.Tensor, y: torch.Tensor, ws: torch.Tensor,
                      act: int = GC_ACT_NONE, r=None, z=None):
    """y = act(z) + r, z = x W^T + b: w is the flat model in the layer's type;
    x [..., columns], y, r and z [..., rows] of that type."""
    cols, dtype = _layer_cols(plan, layer), _DTYPES[layer.type]
    if not isinstance(x, _Tensor) or x.dim() < 1:
        raise ValueError("x: need a tensor of rows")
    lead = x.shape[:-1]
    wide = (*lead, layer.rows)
    xs, ys = _acts(x, dtype, (*lead, cols), "x"), _acts(y, dtype, wide, "y")
    rs = _ABSENT if r is None else _acts(r, dtype, wide, "r")
    zs = _ABSENT if z is None else _acts(z, dtype, wide, "z")
    args = _dev(w, dtype, plan.n_total, "w"), *xs, x.numel() // cols, int(act), *rs, *zs, *ys, *_ws(ws)
    _call("gc_linear_forward", [t for t in (y, x, w, ws, r, z) if t is not None], plan.handle, ctypes.byref(layer), *args)


def gc_act_grad(dy: torch.Tensor, z: torch.Tensor, act: int, dz: torch.Tensor):
    """dz = dy act'(z), elementwise; dz may be dy or z."""
    if not isinstance(dy, _Tensor) or dy.dtype not in _FLOAT_TYPES or dy.dim() < 1:
        raise ValueError("dy: need an fp32, bf16 or fp16 tensor of rows")
    shape = tuple(dy.shape)
    cols = shape[-1]
    ys, zs, ds = (_acts(t, dy.dtype, shape, name) for t, name in ((dy, "dy"), (z, "z"), (dz, "dz")))
    _call("gc_act_grad", (dz, dy, z), *ys, *zs, int(act), _FLOAT_TYPES[dy.dtype], dy.numel() // cols if cols else 0, cols, *ds)


def gc_linear_grad_input(plan: Plan, layer: gc_linear, w, dz: torch.Tensor, dx, ws: torch.Tensor, a=None,
                         act: int = GC_ACT_NONE, z=None, dzx=None):
    """dx = dz W + a, and dzx = (dz W + a) act'(z); dx or dzx may be None."""
    cols, dtype = _layer_cols(plan, layer), _DTYPES[layer.type]
    if not isinstance(dz, _Tensor) or dz.dim() < 1:
        raise ValueError("dz: need a tensor of rows")
    lead = dz.shape[:-1]
    narrow = (*lead, cols)
    ds = _acts(dz, dtype, (*lead, layer.rows), "dz")
    als, zs, xs, gs = (_ABSENT if t is None else _acts(t, dtype, narrow, name)
                       for t, name in ((a, "a"), (z, "z"), (dx, "dx"), (dzx, "dzx")))
    args = _dev(w, dtype, plan.n_total, "w"), *ds, dz.numel() // layer.rows, *als, int(act), *zs, *xs, *gs, *_ws(ws)
    _call("gc_linear_grad_input", [t for t in (dz, w, ws, a, z, dx, dzx) if t is not None], plan.handle,
          ctypes.byref(layer), *args)


def gc_linear_grad_weight(plan: Plan, layer: gc_linear, dz: torch.Tensor, x: torch.Tensor, g, accumulate: bool,
                          ws: torch.Tensor):
    """dz^T x over (accumulate False) or added to the layer's segment of the
    flat fp32 g, and the sum of dz's rows to its bias' segment."""
    cols, dtype = _layer_cols(plan, layer), _DTYPES[layer.type]
    if not isinstance(x, _Tensor) or x.dim() < 1:
        raise ValueError("x: need a tensor of rows")
    lead = x.shape[:-1]
    ds, xs = _acts(dz, dtype, (*lead, layer.rows), "dz"), _acts(x, dtype, (*lead, cols), "x")
    args = *ds, *xs, x.numel() // cols, _f32(g, plan.n_total, "g"), int(bool(accumulate)), *_ws(ws)
    _call("gc_linear_grad_weight", (g, dz, x, ws), plan.handle, ctypes.byref(layer), *args)


# ---------------------------------------------------------- distillation
def _logits(t, name: str):
    """(pointer, GC_* type, row stride, rows, columns) of logits [..., columns]."""
    if not isinstance(t, _Tensor) or t.dtype not in _FLOAT_TYPES or t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name}: need an fp32, bf16 or fp16 tensor of rows")
    v = t.shape[-1]
    return t.data_ptr(), _FLOAT_TYPES[t.dtype], v if t.is_contiguous() else _row_stride(t, name), t.numel() // v, v


def gc_top_logits(logits: torch.Tensor, idx: torch.Tensor, val, lse=None, temperature: float = 1.0):
    """The idx.shape[-1] first logits of every row, by value and then by
    column: int32 columns and fp32 values; lse: the rows' log-sum-exp at 1 /
    temperature, fp32."""
    ptr, kind, stride, n, vocab = _logits(logits, "logits")
    k = idx.shape[-1] if isinstance(idx, _Tensor) and idx.dim() else 0
    if k < 1 or tuple(idx.shape[:-1]) != tuple(logits.shape[:-1]) or not isinstance(val, _Tensor) or val.shape != idx.shape:
        raise ValueError("idx, val: need the logits' rows by k columns")
    ip, vp = _dev(idx, torch.int32, n * k, "idx"), _f32(val, n * k, "val")
    lp = None if lse is None else _f32(lse, n, "lse")
    _call("gc_top_logits", [t for t in (logits, idx, val, lse) if t is not None], ptr, kind, stride, n, vocab, k,
          float(temperature), ip, vp, lp)


def distill_options(temperature: float = 1.0, kd_weight: float = 1.0, ce_weight: float = 0.0, grad_scale: float = 1.0,
                    tail: bool = False) -> gc_distill_options:
    """tail: the teacher's mass outside its entries is held too (GC_DISTILL_REST)."""
    return gc_distill_options(float(temperature), float(kd_weight), float(ce_weight), float(grad_scale),
                              GC_DISTILL_REST if tail else GC_DISTILL_TOP)


def gc_distill_loss(logits: torch.Tensor, idx: torch.Tensor, t: torch.Tensor, opt: gc_distill_options, loss,
                    dlogits=None, t_lse=None, labels=None, weights=None):
    """The rows' losses against the teacher's entries (idx, t) [..., k], and the
    gradient of their sum times opt.grad_scale; dlogits may be logits."""
    ptr, kind, stride, n, vocab = _logits(logits, "logits")
    lead = tuple(logits.shape[:-1])
    if not isinstance(idx, _Tensor) or not isinstance(t, _Tensor) or idx.dim() < 1 or tuple(idx.shape[:-1]) != lead or t.shape != idx.shape:
        raise ValueError("idx, t: need the logits' rows by k columns")
    id_type, t_type, k = _TOKEN_TYPES.get(idx.dtype), _FLOAT_TYPES.get(t.dtype), idx.shape[-1]
    if id_type is None or t_type is None:
        raise ValueError("idx, t: need int32 or int64, and fp32, bf16 or fp16")
    istride, tstride = (k if u.is_contiguous() else _row_stride(u, "idx, t") for u in (idx, t))
    dp, ds = _ABSENT if dlogits is None else _acts(dlogits, logits.dtype, logits.shape, "dlogits")
    tl, wp = (None if u is None else _f32(u, n, name) for u, name in ((t_lse, "t_lse"), (weights, "weights")))
    lp = None if labels is None else _dev(labels, idx.dtype, n, "labels")
    _call("gc_distill_loss", [u for u in (logits, idx, t, loss, dlogits, t_lse, labels, weights) if u is not None], ptr, kind,
          stride, n, vocab, idx.data_ptr(), id_type, istride, t.data_ptr(), t_type, tstride, k, tl, lp, wp,
          ctypes.byref(opt), _f32(loss, n, "loss"), dp, ds)
