"""Python binding of libmoe_b200.so (argument marshalling only).

Every name mirrors an entry point of include/moe_b200.h.  Tensors are torch
CUDA tensors (device memory and streams come from PyTorch); host-side inputs
of the load calls may also be numpy arrays.  There is no fallback: if the
library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_b200.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_STATE, MOE_ERR_OOM, MOE_ERR_CUDA, MOE_ERR_TIMEOUT = range(7)
QUANT = {"int4": 0, "int2": 1, "nvfp4": 2, "bf16": 3, "int4g32": 4, "fp8": 5, "fp6": 6}
SHARED = -1


SCORE = {"softmax": 0, "sigmoid": 1}
GROUP_SCORE = {"max": 0, "top2": 1}
GATE = {"none": 0, "channel": 1, "token": 2, "element": 3}


class MoeError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"[{status}] {msg}")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("hidden", "inter", "num_experts", "top_k", "quant", "has_shared", "max_tokens", "device")]


class QMatrix(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("global_scale", ctypes.c_float)]


class ExpertWeights(ctypes.Structure):
    _fields_ = [("gate", QMatrix), ("up", QMatrix), ("down", QMatrix)]


class RoutingRule(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("num_groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("renorm", ctypes.c_int32), ("scale", ctypes.c_float),
                ("bias", ctypes.c_void_p)]


class AdapterSet(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("ranks", ctypes.c_void_p),
                ("num_adapters", ctypes.c_int32), ("R", ctypes.c_int32), ("K", ctypes.c_int32), ("N", ctypes.c_int32)]


class Norm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("r", "y", "w_post", "gate", "w_pre", "r_out", "x_out")] + \
               [(n, ctypes.c_int64) for n in ("ld_r", "ld_y", "ld_gate", "ld_r_out", "ld_x")] + \
               [(n, ctypes.c_int32) for n in ("T", "H", "r_fp32", "gate_kind", "gate_sigmoid", "unit_offset")] + \
               [(n, ctypes.c_float) for n in ("eps", "branch_scale", "residual_scale")]


class Block(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("r", "x", "y", "x_next", "w_in", "w_post", "w_next", "gate", "logits",
                                               "topk_ids", "topk_w", "adapter_ids")] + \
               [("router_adapters", ctypes.POINTER(AdapterSet)), ("layer_adapters", ctypes.POINTER(AdapterSet))] + \
               [(n, ctypes.c_int32) for n in ("T", "r_fp32", "gate_kind", "gate_sigmoid", "unit_offset")] + \
               [(n, ctypes.c_float) for n in ("eps", "branch_scale", "residual_scale")]


_lib = None


def lib():
    """Load the CUDA library once; raise if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with python -m bit_quantized_mixture_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        sig = {
            "moe_create": [ctypes.POINTER(Config), ctypes.POINTER(vp)],
            "moe_destroy": [vp],
            "moe_load_router": [vp, vp, vp],
            "moe_load_expert_weights": [vp, i32, ctypes.POINTER(ExpertWeights), vp],
            "moe_set_act_global_scales": [vp, f32, f32],
            "moe_route": [vp, vp, i32, vp, vp, vp, vp],
            "moe_route_from_logits": [vp, vp, i32, vp, vp, vp],
            "moe_forward": [vp, vp, i32, vp, vp, vp, vp],
            "moe_route_forward": [vp, vp, i32, vp, vp, vp, vp],
            "moe_quantize": [i32, vp, i32, i32, f32, vp, vp, vp, vp],
            "moe_absmax": [vp, i64, vp, vp],
            "moe_quantize_act_nvfp4": [vp, i32, i32, f32, vp, vp, vp],
            "moe_permute": [vp, i32, i32, i32, vp, vp, vp, vp, vp],
            "moe_debug_unpack_matrix": [vp, i32, i32, vp, vp, vp, vp, vp],
            "moe_set_profile_events": [vp, ctypes.POINTER(vp), i32],
            "moe_sync_status": [vp, vp],
            "moe_permute_noalloc": [vp, i32, i32, i32, vp, vp, vp, vp, vp],
            "moe_expert_block_bytes": [vp, ctypes.POINTER(ctypes.c_size_t)],
            "moe_set_decode_path": [vp, i32],
            "moe_export_expert": [vp, i32, vp, vp],
            "moe_set_expert_table": [vp, ctypes.POINTER(vp), vp],
            "moe_debug_get_permutation": [vp, vp, vp, vp, vp, vp],
            "moe_debug_get_act_nvfp4": [vp, vp, vp, vp],
            "moe_debug_set_wait_test": [vp, i32, i64],
            "moe_select_experts": [vp, i64, i32, i32, i32, ctypes.POINTER(RoutingRule), vp, vp, vp],
            "moe_set_routing": [vp, ctypes.POINTER(RoutingRule), vp],
            "moe_add_adapters": [vp, i64, vp, i64, vp, i64, i32, i32, vp, ctypes.POINTER(AdapterSet), vp],
            "moe_adapters_status": [vp],
            "moe_debug_set_adapter_wait_test": [i32, i64],
            "moe_block_norm": [ctypes.POINTER(Norm), vp],
            "moe_block_forward": [vp, ctypes.POINTER(Block), vp],
            "moe_mma_peak_loop": [i32, i32, i64, vp, ctypes.POINTER(ctypes.c_double), vp],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.moe_status_str.argtypes = [ctypes.c_int]
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_last_error.argtypes = [vp]
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_nvfp4_global_scale.argtypes = [f32]
        L.moe_nvfp4_global_scale.restype = f32
        _lib = L
    return _lib


def _check(status, handle=None):
    if status != MOE_OK:
        raise MoeError(status, lib().moe_last_error(handle).decode())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return t.data_ptr()
    if isinstance(t, np.ndarray):
        assert t.flags["C_CONTIGUOUS"]
        return t.ctypes.data
    raise TypeError(type(t))


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _refuse(msg):
    raise MoeError(MOE_ERR_INVALID_ARG, msg)


_BF16 = (torch.bfloat16,)
_BF16_F32 = (torch.bfloat16, torch.float32)


def _cuda(name, t, dtype, shape, dev):
    """The address of a contiguous tensor of this dtype and shape on device
    number dev (None: any CUDA device)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or \
            (not t.is_cuda if dev is None else t.get_device() != dev):
        _refuse(f"{name}: need a contiguous {dtype} tensor {list(shape)} on " + ("a CUDA device" if dev is None else f"cuda:{dev}"))
    return t.data_ptr()


def _rows(name, t, dtypes, T, W, dev):
    """(address, elements between rows) of a tensor [T, W] on device number dev
    whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.get_device() != dev or t.shape != (T, W):
        _refuse(f"{name}: need {' or '.join(str(d) for d in dtypes)} [{T}, {W}] on cuda:{dev}")
    s0, s1 = t.stride()
    if s1 != 1 and W > 1:
        _refuse(f"{name}: the elements of a row must be contiguous")
    return t.data_ptr(), s0 if T > 1 else W


def _raw(stream):
    """A stream object's (or raw) handle; None stays None: torch's current stream."""
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


_ext = None


def binding():
    """The Python extension with the tensor checks of the calls below; raise if
    it is not built."""
    global _ext
    if _ext is None:
        lib()
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError("_binding.so is missing: build it with python -m bit_quantized_mixture_b200.build") from e
        _binding.init(MoeError)
        _ext = _binding
    return _ext


def _new(shape, dtype, dev, stream):
    """An output tensor; with a stream of its own it belongs to that stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


class Routing:
    """A routing rule (moe_routing): scores, selection bias (fp32 [E] CUDA
    tensor, kept alive here), groups, renormalisation and scale."""

    def __init__(self, score="softmax", bias=None, num_groups=1, top_groups=1, group_score="max", renorm=True, scale=1.0):
        if score not in SCORE or group_score not in GROUP_SCORE:
            _refuse(f"Routing: score must be one of {list(SCORE)}, group_score one of {list(GROUP_SCORE)}")
        if bias is not None and bias.dim() != 1:
            _refuse("Routing: bias must be [E]")
        self._bias = bias
        self.E = None if bias is None else bias.shape[0]
        self.c = RoutingRule(SCORE[score], num_groups, top_groups, GROUP_SCORE[group_score], int(bool(renorm)), scale,
                             _cuda("bias", bias, torch.float32, (self.E,), None) if bias is not None else None)
        self.address = ctypes.addressof(self.c)

    @property
    def bias(self):
        """The bias that the rule was made with (its address is in the rule: a
        new bias needs a new Routing, or is copied into this tensor)."""
        return self._bias


def _device(name, t):
    """The device number of a CUDA tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _refuse(f"{name}: need a CUDA tensor")
    return t.get_device()


def select_experts(logits, k, rule, ids=None, w=None, stream=None):
    """fp32 logits [T, E] -> (ids int32 [T, k], weights fp32 [T, k]) under a
    Routing rule (moe_select_experts)."""
    if ids is None:
        ids = _new((logits.shape[0], k), torch.int32, _device("logits", logits), stream)
    if w is None:
        w = _new((logits.shape[0], k), torch.float32, _device("logits", logits), stream)
    binding().select_experts(logits, k, rule.address, rule.bias, ids, w, _raw(stream))
    return ids, w


def _adapter_set(a, b, scales, ranks, dev):
    if not isinstance(a, torch.Tensor) or a.dim() != 3 or not isinstance(b, torch.Tensor) or b.dim() != 3:
        _refuse("a and b: need [n, R, K] and [n, N, R]")
    n, R, K = a.shape
    N = b.shape[1]
    return AdapterSet(_cuda("a", a, torch.bfloat16, (n, R, K), dev), _cuda("b", b, torch.bfloat16, (n, N, R), dev),
                      _cuda("scales", scales, torch.float32, (n,), dev),
                      None if ranks is None else _cuda("ranks", ranks, torch.int32, (n,), dev), n, R, K, N)


def add_adapters(x, y, adapter_ids, a, b, scales, ranks=None, out=None, stream=None):
    """out_t = y_t + scales[i] b_i (a_i x_t), i = adapter_ids[t]
    (moe_add_adapters): x bf16 [T, K], y bf16 or fp32 [T, N], a bf16
    [n, R, K], b bf16 [n, N, R], scales fp32 [n], ranks int32 [n] or None.
    out may be y; by default it is a new tensor."""
    if out is None:
        out = _new(tuple(y.shape), y.dtype, _device("y", y), stream)
    binding().add_adapters(x, y, adapter_ids, a, b, scales, ranks, out, _raw(stream))
    return out


def adapters_status(stream=None):
    """Synchronize the stream; raise when an add_adapters call on the current
    device gave up a bounded wait since this was last asked for this stream
    (moe_adapters_status)."""
    _check(lib().moe_adapters_status(_stream(stream)))


def debug_set_adapter_wait_test(withhold_cta, wait_limit_cycles=0):
    """Test hook (moe_debug_set_adapter_wait_test): the next launch of the adapters'
    tcgen05 kernel withholds an arrival; its waits give up after the limit."""
    _check(lib().moe_debug_set_adapter_wait_test(int(withhold_cta), int(wait_limit_cycles)))


def _gate(gate, T, H, dev):
    """(kind, address, elements between rows) of a gate tensor by its shape."""
    if gate is None:
        return 0, 0, 0
    if gate.dim() == 2:
        return (GATE["element"],) + _rows("gate", gate, _BF16, T, H, dev)
    if gate.dtype is torch.float32:
        return GATE["token"], _cuda("gate", gate, torch.float32, (T,), dev), 0
    return GATE["channel"], _cuda("gate", gate, torch.bfloat16, (H,), dev), 0


def block_norm(r, y=None, post_weight=None, gate=None, gate_sigmoid=False, pre_weight=None, eps=1e-6, branch_scale=1.0,
               residual_scale=1.0, unit_offset=False, r_out=None, x_out=None, stream=None):
    """The norms, gate and residual add between two blocks (moe_block_norm):
    r bf16 or fp32 [T, H], y bf16 [T, H], weights bf16 [H]; gate bf16 [H]
    (channel), fp32 [T] (token) or bf16 [T, H] (element).  Returns (r', x);
    x is None without pre_weight.  r_out may be r, x_out may be y."""
    if r_out is None:
        r_out = _new(tuple(r.shape), r.dtype, _device("r", r), stream)
    if x_out is None:
        if pre_weight is not None:
            x_out = _new(tuple(r.shape), torch.bfloat16, _device("r", r), stream)
    elif pre_weight is None:
        _refuse("x_out: needs pre_weight")
    binding().block_norm(r, y, post_weight, gate, gate_sigmoid, pre_weight, eps, branch_scale, residual_scale, unit_offset, r_out, x_out,
                         _raw(stream))
    return r_out, x_out


def nvfp4_global_scale(amax: float) -> float:
    return float(lib().moe_nvfp4_global_scale(float(amax)))


class MoeLayer:
    """One MoE layer: owns the weight arena and workspace on one device."""

    def __init__(self, hidden, inter, num_experts, top_k, quant, has_shared, max_tokens, device=0):
        self.cfg = Config(hidden, inter, num_experts, top_k, QUANT[quant], int(bool(has_shared)), max_tokens, device)
        self.quant = quant
        h = ctypes.c_void_p()
        _check(lib().moe_create(ctypes.byref(self.cfg), ctypes.byref(h)))
        self.h = h
        self._keep = []            # host arrays that must outlive asynchronous copies

    def close(self):
        if getattr(self, "h", None):
            lib().moe_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def load_router(self, w_bf16, stream=None):
        _check(lib().moe_load_router(self.h, _ptr(w_bf16), _stream(stream)), self.h)

    def load_expert(self, expert, mats, stream=None):
        """mats: {'gate'|'up'|'down': {'codes', 'scales', 'zeros', 'g'}} arrays in
        interchange layout (torch tensors or numpy arrays)."""
        ew = ExpertWeights()
        for name in ("gate", "up", "down"):
            m = mats[name]
            q = getattr(ew, name)
            q.codes = _ptr(m["codes"])
            q.scales = _ptr(m.get("scales"))
            q.zeros = _ptr(m.get("zeros"))
            q.global_scale = float(m.get("g", 0.0))
        _check(lib().moe_load_expert_weights(self.h, int(expert), ctypes.byref(ew), _stream(stream)), self.h)

    def set_act_global_scales(self, g_x, g_a):
        _check(lib().moe_set_act_global_scales(self.h, float(g_x), float(g_a)), self.h)

    def route(self, x, ids, w, logits=None, stream=None):
        _check(lib().moe_route(self.h, _ptr(x), x.shape[0], _ptr(ids), _ptr(w), _ptr(logits), _stream(stream)), self.h)

    def route_from_logits(self, logits, ids, w, stream=None):
        _check(lib().moe_route_from_logits(self.h, _ptr(logits), logits.shape[0], _ptr(ids), _ptr(w),
                                           _stream(stream)), self.h)

    def forward(self, x, ids, w, y, stream=None):
        _check(lib().moe_forward(self.h, _ptr(x), x.shape[0], _ptr(ids), _ptr(w), _ptr(y), _stream(stream)), self.h)

    def sync_status(self, stream=None):
        """Synchronize the stream; raise on a device-side timeout or CUDA error."""
        _check(lib().moe_sync_status(self.h, _stream(stream)), self.h)

    def route_forward(self, x, ids, w, y, stream=None):
        """The whole layer (route + forward) in one call."""
        _check(lib().moe_route_forward(self.h, _ptr(x), x.shape[0], _ptr(ids), _ptr(w), _ptr(y), _stream(stream)),
               self.h)

    def set_routing(self, rule, stream=None):
        """Follow a Routing rule in route, route_from_logits, route_forward and
        block_forward (None: softmax and top-k again)."""
        if rule is not None and rule.bias is not None and rule.E != self.cfg.num_experts:
            _refuse(f"bias: need {self.cfg.num_experts} entries")
        _check(lib().moe_set_routing(self.h, rule.c if rule is not None else None, _stream(stream)), self.h)
        self._rule = rule          # its bias outlives the asynchronous copy

    def block_forward(self, r, x, y, ids, w, w_in=None, w_post=None, w_next=None, x_next=None, gate=None,
                      gate_sigmoid=False, logits=None, adapter_ids=None, router_adapters=None, layer_adapters=None,
                      eps=1e-6, branch_scale=1.0, residual_scale=1.0, unit_offset=False, stream=None):
        """One MoE block (moe_block_forward): x = norm(r, w_in), the layer x -> y
        with its adapters, r and x_next = block_norm(r, y).  Adapters are
        (a, b, scales, ranks or None) tuples; r is updated in place."""
        dev = self.cfg.device
        H, E, k = self.cfg.hidden, self.cfg.num_experts, self.cfg.top_k
        T = r.shape[0]
        if r.dtype not in _BF16_F32:
            _refuse("r: need bf16 or fp32")
        bf = torch.bfloat16
        b = Block(r=_cuda("r", r, r.dtype, (T, H), dev), x=_cuda("x", x, bf, (T, H), dev), y=_cuda("y", y, bf, (T, H), dev),
                  topk_ids=_cuda("ids", ids, torch.int32, (T, k), dev), topk_w=_cuda("w", w, torch.float32, (T, k), dev),
                  T=T, r_fp32=r.dtype is torch.float32, gate_sigmoid=bool(gate_sigmoid), unit_offset=bool(unit_offset),
                  eps=eps, branch_scale=branch_scale, residual_scale=residual_scale)
        for name, t in (("w_in", w_in), ("w_post", w_post), ("w_next", w_next)):
            if t is not None:
                setattr(b, name, _cuda(name, t, bf, (H,), dev))
        if x_next is not None:
            b.x_next = _cuda("x_next", x_next, bf, (T, H), dev)
        if logits is not None:
            b.logits = _cuda("logits", logits, torch.float32, (T, E), dev)
        b.gate_kind, b.gate, ld_gate = _gate(gate, T, H, dev)
        if b.gate_kind == GATE["element"] and ld_gate != H:
            _refuse("gate: need contiguous rows")
        if adapter_ids is not None:
            b.adapter_ids = _cuda("adapter_ids", adapter_ids, torch.int32, (T,), dev)
        if router_adapters is not None:
            b.router_adapters = ctypes.pointer(_adapter_set(*router_adapters, dev))
        if layer_adapters is not None:
            b.layer_adapters = ctypes.pointer(_adapter_set(*layer_adapters, dev))
        _check(lib().moe_block_forward(self.h, b, _stream(stream)), self.h)

    def set_profile_events(self, events):
        """events: 5 to 10 torch.cuda.Event(enable_timing=True) (recorded once
        beforehand) or None; slot meanings as in moe_set_profile_events."""
        if events is None:
            _check(lib().moe_set_profile_events(self.h, None, 0), self.h)
            return
        arr = (ctypes.c_void_p * len(events))(*[ev.cuda_event for ev in events])
        _check(lib().moe_set_profile_events(self.h, arr, len(events)), self.h)

    def set_decode_path(self, path):
        """'auto' (fused kernel eagerly, three kernels inside a CUDA graph),
        'fused', 'kernels' or 'gemm' (the grouped-GEMM path for every T)."""
        _check(lib().moe_set_decode_path(self.h, {"auto": 0, "fused": 1, "kernels": 2, "gemm": 3}[path]), self.h)

    def expert_block_bytes(self):
        n = ctypes.c_size_t(0)
        _check(lib().moe_expert_block_bytes(self.h, ctypes.byref(n)), self.h)
        return int(n.value)

    def export_expert(self, expert, dst, stream=None):
        """Copy expert `expert`'s block (device layout) to the CUDA buffer dst."""
        _check(lib().moe_export_expert(self.h, int(expert), _ptr(dst), _stream(stream)), self.h)

    def set_expert_table(self, addresses, stream=None):
        """addresses: E device addresses (ints) of expert blocks, or None for the arena."""
        if addresses is None:
            _check(lib().moe_set_expert_table(self.h, None, _stream(stream)), self.h)
            return
        arr = (ctypes.c_void_p * len(addresses))(*[int(a) for a in addresses])
        _check(lib().moe_set_expert_table(self.h, arr, _stream(stream)), self.h)

    def debug_permutation(self, T, stream=None):
        """(counts, offsets, perm, inv) of the last grouped-GEMM forward of T tokens."""
        E, k = self.cfg.num_experts, self.cfg.top_k
        dev = torch.device("cuda", self.cfg.device)
        counts = torch.empty(E, dtype=torch.int32, device=dev)
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        perm = torch.empty(T * k, dtype=torch.int32, device=dev)
        inv = torch.empty(T * k, dtype=torch.int32, device=dev)
        _check(lib().moe_debug_get_permutation(self.h, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv),
                                               _stream(stream)), self.h)
        return counts, offsets, perm, inv

    def debug_act_nvfp4(self, T, stream=None):
        """(codes [T*k, H/2], scales [T*k, H/16]) of the W4A4 operand of the last
        block-scaled NVFP4 grouped-GEMM forward of T tokens, permuted order."""
        slots, H = T * self.cfg.top_k, self.cfg.hidden
        dev = torch.device("cuda", self.cfg.device)
        codes = torch.empty((slots, H // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((slots, H // 16), dtype=torch.uint8, device=dev)
        _check(lib().moe_debug_get_act_nvfp4(self.h, _ptr(codes), _ptr(scales), _stream(stream)), self.h)
        return codes, scales

    def debug_set_wait_test(self, withhold_cta, wait_limit_cycles=0):
        """One-shot test hook: the next fused decode launch has CTA
        withhold_cta skip a grid-barrier arrival, and its waits give up after
        wait_limit_cycles (0: the default limit)."""
        _check(lib().moe_debug_set_wait_test(self.h, int(withhold_cta), int(wait_limit_cycles)), self.h)

    def debug_unpack(self, expert, which, codes, scales=None, zeros=None, global_scale=None, stream=None):
        _check(lib().moe_debug_unpack_matrix(self.h, int(expert), int(which), _ptr(codes), _ptr(scales),
                                             _ptr(zeros), _ptr(global_scale), _stream(stream)), self.h)


def quantize(quant, w, global_scale=0.0, stream=None):
    """w: CUDA fp32 [N, K] -> (codes, scales, zeros) CUDA uint8/fp16 tensors."""
    N, K = w.shape
    dev = w.device
    q = QUANT[quant]
    zeros = None
    if quant in ("int4", "int4g32"):
        codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((N, K // (32 if quant == "int4g32" else 128)), dtype=torch.float16, device=dev)
    elif quant == "fp6":
        codes = torch.empty((N, K), dtype=torch.uint8, device=dev)
        scales = torch.empty((N, K // 32), dtype=torch.float16, device=dev)
    elif quant == "fp8":
        codes = torch.empty((N, K), dtype=torch.uint8, device=dev)
        scales = torch.empty((N // 128, K // 128), dtype=torch.float32, device=dev)
    elif quant == "int2":
        codes = torch.empty((N, K // 4), dtype=torch.uint8, device=dev)
        scales = torch.empty((N, K // 128), dtype=torch.float16, device=dev)
        zeros = torch.empty((N // 4, K // 128), dtype=torch.uint8, device=dev)
    else:
        codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((N, K // 16), dtype=torch.uint8, device=dev)
    _check(lib().moe_quantize(q, _ptr(w), N, K, float(global_scale), _ptr(codes), _ptr(scales), _ptr(zeros),
                              _stream(stream)))
    return codes, scales, zeros


def absmax(x, out, stream=None):
    _check(lib().moe_absmax(_ptr(x), x.numel(), _ptr(out), _stream(stream)))


def quantize_act_nvfp4(x, g, stream=None):
    T, K = x.shape
    codes = torch.empty((T, K // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((T, K // 16), dtype=torch.uint8, device=x.device)
    _check(lib().moe_quantize_act_nvfp4(_ptr(x), T, K, float(g), _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def permute(ids, num_experts, stream=None):
    T, k = ids.shape
    dev = ids.device
    counts = torch.empty(num_experts, dtype=torch.int32, device=dev)
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(T * k, dtype=torch.int32, device=dev)
    inv = torch.empty(T * k, dtype=torch.int32, device=dev)
    _check(lib().moe_permute(_ptr(ids), T, k, num_experts, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv),
                             _stream(stream)))
    return counts, offsets, perm, inv


def permute_noalloc(ids, num_experts, stream=None):
    """moe_permute without device allocation (scratch in a static device array)."""
    T, k = ids.shape
    dev = ids.device
    counts = torch.empty(num_experts, dtype=torch.int32, device=dev)
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(T * k, dtype=torch.int32, device=dev)
    inv = torch.empty(T * k, dtype=torch.int32, device=dev)
    _check(lib().moe_permute_noalloc(_ptr(ids), T, k, num_experts, _ptr(counts), _ptr(offsets), _ptr(perm),
                                     _ptr(inv), _stream(stream)))
    return counts, offsets, perm, inv


def mma_peak_loop(kind, issuers, iters, err, stream=None):
    """Launch the tensor-core throughput loop (kind 0: bf16 kind::f16, 1: e2m1
    block-scaled) on every SM; returns the FLOPs of the launch.  err: a
    zeroed int32 CUDA tensor that receives a code if a wait gave up."""
    flops = ctypes.c_double(0.0)
    _check(lib().moe_mma_peak_loop(int(kind), int(issuers), int(iters), _ptr(err), ctypes.byref(flops),
                                   _stream(stream)))
    return flops.value
