"""Python binding of libling_moe.so, the B200 W4 g32 MoE-layer library.

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels.  The functions below carry the C ABI's names and arguments
(pointers are integers, streams are raw cudaStream_t values); `MoELayer`
wraps them for torch tensors.  The library must have been built
(`python -m weight_only_int4_fp32_b200.build`); the first call into it
raises if it is missing -- there is nothing else to fall back to.
"""
from __future__ import annotations

import ctypes
import os
import struct

__all__ = [
    "LING_MOE_OK", "LING_MOE_ERR_INVALID_ARG", "LING_MOE_ERR_CUDA", "LING_MOE_ERR_OOM",
    "LING_MOE_ERR_UNSUPPORTED", "LING_MOE_ERR_DEVICE_TIMEOUT", "LingMoEError",
    "ling_moe_config_t", "ling_moe_weights_t", "library_path", "load_library",
    "ling_moe_create", "ling_moe_create_mxfp4", "ling_moe_forward", "ling_moe_forward_ex", "ling_moe_forward_host",
    "ling_moe_status", "ling_moe_describe", "ling_moe_launch_count", "ling_moe_last_error",
    "ling_moe_destroy", "ling_moe_test_set_wait", "ling_moe_route_noalloc", "ling_moe_route_noalloc_status",
    "ling_moe_route_noalloc_test_set_wait", "ling_moe_set_kernel_timing",
    "ling_moe_kernel_times", "ling_moe_ep_t", "ling_moe_create_ep", "ling_moe_forward_partial",
    "ling_moe_round_bf16", "LING_MOE_FORMAT_INT4", "LING_MOE_FORMAT_MXFP4", "round_bf16",
    "MoELayer", "LMHeadFP8", "EXPORTED",
    "LING_MOE_TYPE_F32", "LING_MOE_TYPE_BF16", "BeamSearch", "BlockFP8Linear",
    "GatedDeltaRule", "ling_moe_delta_config_t", "ling_moe_delta_io_t",
]

LING_MOE_OK = 0
LING_MOE_ERR_INVALID_ARG = -1
LING_MOE_ERR_CUDA = -2
LING_MOE_ERR_OOM = -3
LING_MOE_ERR_UNSUPPORTED = -4
LING_MOE_ERR_DEVICE_TIMEOUT = -5
LING_MOE_FORMAT_INT4 = 0
LING_MOE_FORMAT_MXFP4 = 1
LING_MOE_TYPE_F32 = 0
LING_MOE_TYPE_BF16 = 1

# every symbol include/ling_moe.h declares
EXPORTED = (
    "ling_moe_create", "ling_moe_create_mxfp4", "ling_moe_forward", "ling_moe_forward_ex",
    "ling_moe_forward_host", "ling_moe_status", "ling_moe_describe", "ling_moe_launch_count",
    "ling_moe_last_error", "ling_moe_destroy", "ling_moe_test_set_wait", "ling_moe_route_noalloc",
    "ling_moe_route_noalloc_status", "ling_moe_route_noalloc_test_set_wait", "ling_moe_set_kernel_timing",
    "ling_moe_kernel_times", "ling_moe_kernel_name", "ling_moe_create_ep", "ling_moe_forward_partial",
    "ling_moe_round_bf16",
    "ling_moe_lmhead_create", "ling_moe_lmhead_forward", "ling_moe_lmhead_forward_ex",
    "ling_moe_lmhead_forward_host", "ling_moe_lmhead_weights", "ling_moe_lmhead_status",
    "ling_moe_lmhead_launch_count", "ling_moe_lmhead_destroy", "ling_moe_lmhead_test_set_wait",
    "ling_moe_beam_create", "ling_moe_beam_select", "ling_moe_beam_reorder", "ling_moe_beam_launch_count",
    "ling_moe_beam_destroy",
    "ling_moe_fp8_linear_create", "ling_moe_fp8_linear_forward", "ling_moe_fp8_linear_status",
    "ling_moe_fp8_linear_launch_count", "ling_moe_fp8_linear_destroy", "ling_moe_fp8_linear_test_set_wait",
    "ling_moe_delta_create", "ling_moe_delta_step", "ling_moe_delta_prefill", "ling_moe_delta_status",
    "ling_moe_delta_launch_count", "ling_moe_delta_destroy", "ling_moe_delta_test_set_wait",
)

_HERE = os.path.dirname(os.path.abspath(__file__))


def library_path() -> str:
    return os.environ.get("LING_MOE_LIB", os.path.join(_HERE, "libling_moe.so"))


class LingMoEError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"ling_moe error {code}: {msg}")
        self.code = code


class ling_moe_config_t(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("inter", ctypes.c_int), ("num_experts", ctypes.c_int),
                ("top_k", ctypes.c_int), ("group_size", ctypes.c_int), ("max_tokens", ctypes.c_int)]


class ling_moe_weights_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "router_w", "router_bias", "gate_q", "gate_s", "up_q", "up_s", "down_q", "down_s",
        "sh_gate", "sh_up", "sh_down")]


class ling_moe_ep_t(ctypes.Structure):
    _fields_ = [("expert_begin", ctypes.c_int), ("expert_count", ctypes.c_int), ("with_shared", ctypes.c_int),
                ("format", ctypes.c_int)]


class ling_moe_delta_config_t(ctypes.Structure):
    _fields_ = [("k_heads", ctypes.c_int), ("v_heads", ctypes.c_int), ("head_k", ctypes.c_int),
                ("head_v", ctypes.c_int), ("max_tokens", ctypes.c_int), ("max_seqs", ctypes.c_int),
                ("scale", ctypes.c_float)]


class ling_moe_delta_io_t(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v", "g", "beta")]
                + [(n + "_stride", ctypes.c_int64 * 3) for n in ("q", "k", "v", "g", "beta")]
                + [("g_channel_stride", ctypes.c_int64), ("out", ctypes.c_void_p), ("state", ctypes.c_void_p),
                   ("num_slots", ctypes.c_int), ("slots", ctypes.c_void_p)])


_LIB = None


def load_library():
    """Load libling_moe.so once (raises ImportError if it is missing or stale)."""
    global _LIB
    if _LIB is None:
        _LIB = _load()
    return _LIB


def _load():
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(
            f"libling_moe.so not found at {path}: build it with "
            "`python -m weight_only_int4_fp32_b200.build` (there is no fallback path)")
    L = ctypes.CDLL(path)
    vp, ci, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    sig = {
        "ling_moe_create": (ci, [ctypes.POINTER(ling_moe_config_t), ctypes.POINTER(ling_moe_weights_t),
                                 ctypes.POINTER(vp)]),
        "ling_moe_create_mxfp4": (ci, [ctypes.POINTER(ling_moe_config_t), ctypes.POINTER(ling_moe_weights_t),
                                       ctypes.POINTER(vp)]),
        "ling_moe_create_ep": (ci, [ctypes.POINTER(ling_moe_config_t), ctypes.POINTER(ling_moe_weights_t),
                                    ctypes.POINTER(ling_moe_ep_t), ctypes.POINTER(vp)]),
        "ling_moe_forward_partial": (ci, [vp, vp, ci, vp, vp, vp, vp]),
        "ling_moe_round_bf16": (ci, [vp, vp, ctypes.c_size_t, vp]),
        "ling_moe_forward": (ci, [vp, vp, ci, vp, vp]),
        "ling_moe_forward_ex": (ci, [vp, vp, ci, vp, vp, vp, vp]),
        "ling_moe_forward_host": (ci, [vp, vp, ci, vp, vp]),
        "ling_moe_status": (ci, [vp, vp]),
        "ling_moe_describe": (ctypes.c_char_p, [vp]),
        "ling_moe_launch_count": (i64, [vp]),
        "ling_moe_last_error": (ctypes.c_char_p, []),
        "ling_moe_destroy": (None, [vp]),
        "ling_moe_test_set_wait": (ci, [vp, ci, ctypes.c_uint64]),
        "ling_moe_route_noalloc": (ci, [vp, ci, vp, vp, ci, ci, vp, vp, vp]),
        "ling_moe_route_noalloc_status": (ci, [vp]),
        "ling_moe_route_noalloc_test_set_wait": (ci, [ci, ctypes.c_uint64]),
        "ling_moe_set_kernel_timing": (ci, [vp, ci]),
        "ling_moe_kernel_times": (ci, [vp, ctypes.POINTER(ctypes.c_float), ci, ctypes.POINTER(ci)]),
        "ling_moe_kernel_name": (ctypes.c_char_p, [vp, ci]),
        "ling_moe_lmhead_create": (ci, [vp, ci, ci, ctypes.POINTER(vp)]),
        "ling_moe_lmhead_forward": (ci, [vp, vp, ci, vp, vp]),
        "ling_moe_lmhead_forward_ex": (ci, [vp, vp, ci, vp, vp, vp, vp]),
        "ling_moe_lmhead_forward_host": (ci, [vp, vp, ci, vp, vp]),
        "ling_moe_lmhead_weights": (ci, [vp, vp, vp, vp]),
        "ling_moe_lmhead_status": (ci, [vp, vp]),
        "ling_moe_lmhead_launch_count": (i64, [vp]),
        "ling_moe_lmhead_destroy": (None, [vp]),
        "ling_moe_lmhead_test_set_wait": (ci, [vp, ci, ctypes.c_uint64]),
        "ling_moe_beam_create": (ci, [ci, ci, ci, ctypes.POINTER(vp)]),
        "ling_moe_beam_select": (ci, [vp, vp, ci, i64, i64, ci, vp, vp, ci, vp, vp, vp, vp, vp]),
        "ling_moe_beam_reorder": (ci, [ctypes.POINTER(vp), ctypes.POINTER(ctypes.c_size_t), ci, ci, vp, vp, ci, ci,
                                       vp]),
        "ling_moe_beam_launch_count": (i64, [vp]),
        "ling_moe_beam_destroy": (None, [vp]),
        "ling_moe_delta_create": (ci, [ctypes.POINTER(ling_moe_delta_config_t), ctypes.POINTER(vp)]),
        "ling_moe_delta_step": (ci, [vp, vp, ci, ci, vp, vp]),
        "ling_moe_delta_prefill": (ci, [vp, vp, ci, vp, ci, vp, vp]),
        "ling_moe_delta_status": (ci, [vp, vp]),
        "ling_moe_delta_launch_count": (i64, [vp]),
        "ling_moe_delta_destroy": (None, [vp]),
        "ling_moe_delta_test_set_wait": (ci, [vp, ci, ctypes.c_uint64]),
        "ling_moe_fp8_linear_create": (ci, [vp, vp, ci, ci, ci, ctypes.POINTER(vp)]),
        "ling_moe_fp8_linear_forward": (ci, [vp, vp, i64, ci, vp, ci, i64, vp]),
        "ling_moe_fp8_linear_status": (ci, [vp, vp]),
        "ling_moe_fp8_linear_launch_count": (i64, [vp]),
        "ling_moe_fp8_linear_destroy": (None, [vp]),
        "ling_moe_fp8_linear_test_set_wait": (ci, [vp, ci, ctypes.c_uint64]),
    }
    for name, (res, args) in sig.items():
        try:
            f = getattr(L, name)
        except AttributeError as e:
            raise ImportError(f"{path} lacks {name}: rebuild it "
                              "(`python -m weight_only_int4_fp32_b200.build`)") from e
        f.restype = res
        f.argtypes = args
    return L


class _LazyLib:
    def __getattr__(self, name):
        f = getattr(load_library(), name)
        setattr(self, name, f)  # found without this call from now on
        return f


lib = _LazyLib()


def ling_moe_last_error() -> str:
    return lib.ling_moe_last_error().decode()


def _check(rc: int) -> int:
    if rc != LING_MOE_OK:
        raise LingMoEError(rc, ling_moe_last_error())
    return rc


def ling_moe_create(cfg: ling_moe_config_t, weights: ling_moe_weights_t) -> int:
    h = ctypes.c_void_p()
    _check(lib.ling_moe_create(ctypes.byref(cfg), ctypes.byref(weights), ctypes.byref(h)))
    return h.value


def ling_moe_create_mxfp4(cfg: ling_moe_config_t, weights: ling_moe_weights_t) -> int:
    h = ctypes.c_void_p()
    _check(lib.ling_moe_create_mxfp4(ctypes.byref(cfg), ctypes.byref(weights), ctypes.byref(h)))
    return h.value


def ling_moe_create_ep(cfg: ling_moe_config_t, weights: ling_moe_weights_t, ep: ling_moe_ep_t) -> int:
    h = ctypes.c_void_p()
    _check(lib.ling_moe_create_ep(ctypes.byref(cfg), ctypes.byref(weights), ctypes.byref(ep), ctypes.byref(h)))
    return h.value


def ling_moe_forward_partial(h: int, x: int, T: int, partial: int, topk_idx: int = None, topk_w: int = None,
                             stream: int = 0) -> int:
    return _check(lib.ling_moe_forward_partial(h, x, T, partial, topk_idx, topk_w, stream))


def ling_moe_round_bf16(inp: int, out: int, n: int, stream: int = 0) -> int:
    return _check(lib.ling_moe_round_bf16(inp, out, n, stream))


def ling_moe_set_kernel_timing(h: int, on: bool) -> int:
    return _check(lib.ling_moe_set_kernel_timing(h, 1 if on else 0))


def ling_moe_kernel_times(h: int) -> list:
    """[(kernel name, ms)] of the last forward call issued with timing on."""
    ms = (ctypes.c_float * 16)()
    n = ctypes.c_int(0)
    _check(lib.ling_moe_kernel_times(h, ms, 16, ctypes.byref(n)))
    return [(lib.ling_moe_kernel_name(h, i).decode(), float(ms[i])) for i in range(n.value)]


def ling_moe_forward(h: int, x: int, T: int, out: int, stream: int = 0) -> int:
    return _check(lib.ling_moe_forward(h, x, T, out, stream))


def ling_moe_forward_ex(h: int, x: int, T: int, out: int, topk_idx: int, topk_w: int,
                        stream: int = 0) -> int:
    return _check(lib.ling_moe_forward_ex(h, x, T, out, topk_idx, topk_w, stream))


def ling_moe_forward_host(h: int, x_host: int, T: int, out_host: int, stream: int = 0) -> int:
    return _check(lib.ling_moe_forward_host(h, x_host, T, out_host, stream))


def ling_moe_status(h: int, stream: int = 0) -> int:
    """Returns the status code (does not raise on DEVICE_TIMEOUT)."""
    return lib.ling_moe_status(h, stream)


def ling_moe_describe(h: int) -> str:
    return lib.ling_moe_describe(h).decode()


def ling_moe_launch_count(h: int) -> int:
    return lib.ling_moe_launch_count(h)


def ling_moe_destroy(h: int) -> None:
    lib.ling_moe_destroy(h)


def ling_moe_test_set_wait(h: int, skip_arrive_cta: int, wait_limit_ns: int) -> int:
    return _check(lib.ling_moe_test_set_wait(h, skip_arrive_cta, wait_limit_ns))


def ling_moe_route_noalloc(x: int, T: int, router_w: int, router_bias, num_experts: int, top_k: int,
                           topk_idx: int, topk_w: int, stream: int = 0) -> int:
    """Routing with the library's static scratch; allocates nothing (see ling_moe.h)."""
    return _check(lib.ling_moe_route_noalloc(x, T, router_w, router_bias or None, num_experts, top_k,
                                             topk_idx, topk_w, stream))


def ling_moe_route_noalloc_status(stream: int = 0) -> int:
    """LING_MOE_OK, or LING_MOE_ERR_DEVICE_TIMEOUT if a routing wait gave up since the last check
    (returned, not raised, like MoELayer.status)."""
    rc = lib.ling_moe_route_noalloc_status(stream)
    if rc not in (LING_MOE_OK, LING_MOE_ERR_DEVICE_TIMEOUT):
        raise LingMoEError(rc, ling_moe_last_error())
    return rc


def ling_moe_route_noalloc_test_set_wait(skip_cta: int, wait_limit_ns: int) -> int:
    return _check(lib.ling_moe_route_noalloc_test_set_wait(skip_cta, wait_limit_ns))


def _require(t, shape, dtype, cuda: bool, name: str):
    """Raise ValueError unless t is a contiguous tensor of this shape and dtype
    on the GPU (cuda) or the host; the C calls trust the sizes they are given."""
    if (t.shape != tuple(shape) or t.dtype != dtype or t.is_cuda != cuda
            or not t.is_contiguous()):
        where = "CUDA" if cuda else "host"
        raise ValueError(f"{name} must be a contiguous {where} {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def round_bf16(partial, out=None, stream=None):
    """bf16 round-to-nearest-even of an fp32 CUDA tensor (ling_moe_round_bf16):
    the last step of an expert-parallel combine."""
    import torch
    if not partial.is_cuda or partial.dtype != torch.float32 or not partial.is_contiguous():
        raise ValueError("partial must be a contiguous CUDA float32 tensor")
    if out is None:
        out = torch.empty(partial.shape, dtype=torch.bfloat16, device=partial.device)
    _require(out, tuple(partial.shape), torch.bfloat16, True, "out")
    s = torch.cuda.current_stream().cuda_stream if stream is None else getattr(stream, "cuda_stream", stream)
    ling_moe_round_bf16(partial.data_ptr(), out.data_ptr(), partial.numel(), s)
    return out


class MoELayer:
    """One MoE layer on the current CUDA device, built from torch tensors.

    `weights` maps the canonical names (router_w, router_bias, gate_q, gate_s,
    up_q, up_s, down_q, down_s, sh_gate, sh_up, sh_down) to contiguous CUDA
    tensors; they are copied, so they may be freed after construction.
    fmt="int4" (W4 g32, bf16 scales) or "mxfp4" (E2M1 codes, E8M0 scale bytes).
    """

    def __init__(self, weights: dict, top_k: int = 8, max_tokens: int = 1, group_size: int = 32,
                 fmt: str = "int4", ep: tuple | None = None):
        """ep = (expert_begin, expert_count, with_shared): an expert-parallel
        handle (ling_moe_create_ep) whose routed weights hold only experts
        [expert_begin, expert_begin + expert_count) of the router's E; it
        serves forward_partial only."""
        import torch  # device memory and streams only
        rw = weights["router_w"]
        E, H = rw.shape
        I = (weights["sh_gate"] if weights.get("sh_gate") is not None else weights["gate_q"][0]).shape[0]
        for k, v in weights.items():
            if v is not None and (not v.is_cuda or not v.is_contiguous()):
                raise ValueError(f"{k} must be a contiguous CUDA tensor")
        cfg = ling_moe_config_t(H, I, E, top_k, group_size, max_tokens)
        ptr = lambda n: (weights[n].data_ptr() if weights.get(n) is not None else None)
        w = ling_moe_weights_t(*(ptr(n) for n, _ in ling_moe_weights_t._fields_))
        self.E, self.H, self.I, self.k, self.max_tokens = E, H, I, top_k, max_tokens
        if fmt not in ("int4", "mxfp4"):
            raise ValueError("fmt must be 'int4' or 'mxfp4'")
        self.ep = ep
        if ep is not None:
            b, n, sh = ep
            spec = ling_moe_ep_t(int(b), int(n), int(bool(sh)),
                                 LING_MOE_FORMAT_MXFP4 if fmt == "mxfp4" else LING_MOE_FORMAT_INT4)
            self.handle = ling_moe_create_ep(cfg, w, spec)
        else:
            self.handle = (ling_moe_create_mxfp4 if fmt == "mxfp4" else ling_moe_create)(cfg, w)
        self._torch = torch

    def _stream(self, stream):
        if stream is None:
            return self._torch.cuda.current_stream().cuda_stream
        return getattr(stream, "cuda_stream", stream)

    def forward(self, x, out=None, stream=None, return_routing: bool = False):
        torch = self._torch
        if x.dim() != 2:
            raise ValueError("x must be 2-D [T, hidden]")
        T = x.shape[0]
        _require(x, (T, self.H), torch.bfloat16, True, "x")
        if out is None:
            out = torch.empty_like(x)
        _require(out, (T, self.H), torch.bfloat16, True, "out")
        s = self._stream(stream)
        if return_routing:
            idx = torch.empty((T, self.k), dtype=torch.int32, device=x.device)
            w = torch.empty((T, self.k), dtype=torch.float32, device=x.device)
            ling_moe_forward_ex(self.handle, x.data_ptr(), T, out.data_ptr(), idx.data_ptr(),
                                w.data_ptr(), s)
            return out, idx, w
        ling_moe_forward(self.handle, x.data_ptr(), T, out.data_ptr(), s)
        return out

    __call__ = forward

    def forward_partial(self, x, out=None, stream=None, return_routing: bool = False):
        """fp32 [T, hidden]: the sum of the terms this handle computes (all of
        the layer on an ordinary handle), before the bf16 rounding."""
        torch = self._torch
        if x.dim() != 2:
            raise ValueError("x must be 2-D [T, hidden]")
        T = x.shape[0]
        _require(x, (T, self.H), torch.bfloat16, True, "x")
        if out is None:
            out = torch.empty((T, self.H), dtype=torch.float32, device=x.device)
        _require(out, (T, self.H), torch.float32, True, "out")
        s = self._stream(stream)
        idx = w = None
        if return_routing:
            idx = torch.empty((T, self.k), dtype=torch.int32, device=x.device)
            w = torch.empty((T, self.k), dtype=torch.float32, device=x.device)
        ling_moe_forward_partial(self.handle, x.data_ptr(), T, out.data_ptr(),
                                 idx.data_ptr() if idx is not None else None,
                                 w.data_ptr() if w is not None else None, s)
        return (out, idx, w) if return_routing else out

    def forward_host(self, x_host, out_host=None, stream=None):
        torch = self._torch
        T = x_host.shape[0]
        _require(x_host, (T, self.H), torch.bfloat16, False, "x_host")
        if out_host is None:
            out_host = torch.empty_like(x_host)
        _require(out_host, (T, self.H), torch.bfloat16, False, "out_host")
        ling_moe_forward_host(self.handle, x_host.data_ptr(), T, out_host.data_ptr(), self._stream(stream))
        return out_host

    def status(self, stream=None) -> int:
        return ling_moe_status(self.handle, self._stream(stream))

    def describe(self) -> str:
        return ling_moe_describe(self.handle)

    def launch_count(self) -> int:
        return ling_moe_launch_count(self.handle)

    def set_kernel_timing(self, on: bool = True):
        ling_moe_set_kernel_timing(self.handle, on)

    def kernel_times(self) -> list:
        """[(kernel name, ms)] of the last forward call issued with timing on."""
        return ling_moe_kernel_times(self.handle)

    def close(self):
        if getattr(self, "handle", None):
            ling_moe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class LMHeadFP8:
    """The online-FP8 LM head on the current CUDA device.

    `w` is the bf16 head [vocab, hidden] (contiguous CUDA tensor); it is
    quantised to e4m3 with one fp32 scale per row when the object is built
    and may be freed afterwards.  Each call quantises its tokens the same
    way and returns fp32 logits [T, vocab] (T <= 8).
    """

    MAX_TOKENS = 8

    def __init__(self, w):
        import torch  # device memory and streams only
        if w.dtype != torch.bfloat16 or not w.is_cuda or not w.is_contiguous() or w.dim() != 2:
            raise ValueError("w must be a contiguous 2-D bf16 CUDA tensor")
        self.vocab, self.hidden = w.shape
        h = ctypes.c_void_p()
        _check(lib.ling_moe_lmhead_create(w.data_ptr(), self.vocab, self.hidden, ctypes.byref(h)))
        self.handle = h.value
        self._torch = torch

    def _stream(self, stream):
        if stream is None:
            return self._torch.cuda.current_stream().cuda_stream
        return getattr(stream, "cuda_stream", stream)

    def forward(self, x, logits=None, stream=None, return_codes: bool = False):
        torch = self._torch
        if x.dim() != 2:
            raise ValueError("x must be 2-D [T, hidden]")
        T = x.shape[0]
        _require(x, (T, self.hidden), torch.bfloat16, True, "x")
        if logits is None:
            logits = torch.empty((T, self.vocab), dtype=torch.float32, device=x.device)
        _require(logits, (T, self.vocab), torch.float32, True, "logits")
        s = self._stream(stream)
        if return_codes:
            xq = torch.empty((T, self.hidden), dtype=torch.uint8, device=x.device)
            xs = torch.empty((T,), dtype=torch.float32, device=x.device)
            _check(lib.ling_moe_lmhead_forward_ex(self.handle, x.data_ptr(), T, logits.data_ptr(),
                                                  xq.data_ptr(), xs.data_ptr(), s))
            return logits, xq, xs
        _check(lib.ling_moe_lmhead_forward(self.handle, x.data_ptr(), T, logits.data_ptr(), s))
        return logits

    __call__ = forward

    def forward_host(self, x_host, logits_host=None, stream=None):
        torch = self._torch
        T = x_host.shape[0]
        _require(x_host, (T, self.hidden), torch.bfloat16, False, "x_host")
        if logits_host is None:
            logits_host = torch.empty((T, self.vocab), dtype=torch.float32, pin_memory=True)
        _require(logits_host, (T, self.vocab), torch.float32, False, "logits_host")
        _check(lib.ling_moe_lmhead_forward_host(self.handle, x_host.data_ptr(), T, logits_host.data_ptr(),
                                                self._stream(stream)))
        return logits_host

    def weights(self, stream=None):
        """(codes uint8 [vocab, hidden], scales fp32 [vocab]): the handle's quantised head, row-major."""
        torch = self._torch
        codes = torch.empty((self.vocab, self.hidden), dtype=torch.uint8, device="cuda")
        scales = torch.empty((self.vocab,), dtype=torch.float32, device="cuda")
        _check(lib.ling_moe_lmhead_weights(self.handle, codes.data_ptr(), scales.data_ptr(), self._stream(stream)))
        return codes, scales

    def status(self, stream=None) -> int:
        """Status code of the handle's device work (does not raise on DEVICE_TIMEOUT)."""
        return lib.ling_moe_lmhead_status(self.handle, self._stream(stream))

    def launch_count(self) -> int:
        return lib.ling_moe_lmhead_launch_count(self.handle)

    def test_set_wait(self, skip_cta: int, wait_limit_ns: int = 0):
        """Test hook (see ling_moe_lmhead_test_set_wait)."""
        _check(lib.ling_moe_lmhead_test_set_wait(self.handle, skip_cta, wait_limit_ns))

    def close(self):
        if getattr(self, "handle", None):
            lib.ling_moe_lmhead_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _raw_stream(torch, stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return getattr(stream, "cuda_stream", stream)


def _on_current_device(torch, name, *tensors):
    """The library launches on the current device: its tensors have to live there."""
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != cur:
            raise ValueError(f"{name}: a tensor on {t.device}, the current device is cuda:{cur}")


def _new(torch, like, shape, dtype, stream):
    """An output tensor on `like`'s device (shape None: like's own), whose memory belongs to the stream that
    writes it: on another one, memory that the current stream has just given back could still be in use."""
    if stream is not None:
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream)
        with torch.cuda.stream(s):
            return _new(torch, like, shape, dtype, None)
    if shape is None:  # the quickest call
        return torch.empty_like(like, dtype=dtype)
    return like.new_empty(shape, dtype=dtype)


class _Handle:
    """A library handle that is freed with its object."""

    _destroy = None  # name of the C call

    def close(self):
        if getattr(self, "handle", None):
            getattr(lib, self._destroy)(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BeamSearch(_Handle):
    """Beam search for up to `max_groups` requests of `beams` beams each over `vocab` tokens.

    `select` takes one step's logits (LMHeadFP8's, or any) and the beams'
    accumulated scores to the next beams; `reorder` moves the beams' states
    to their new places.  Definitions and limits: ling_moe_beam_select and
    ling_moe_beam_reorder in ling_moe.h.
    """

    _destroy = "ling_moe_beam_destroy"

    def __init__(self, max_groups: int, beams: int, vocab: int):
        import torch  # device memory and streams only
        self.max_groups, self.beams, self.vocab = int(max_groups), int(beams), int(vocab)
        h = ctypes.c_void_p()
        _check(lib.ling_moe_beam_create(self.max_groups, self.beams, self.vocab, ctypes.byref(h)))
        self.handle = h.value
        self._torch = torch

    def select(self, logits, scores, finished=None, eos: int = -1, stream=None):
        """(tokens int32, parents int32, scores fp32, finished bool), each [groups, beams], best first.

        logits: fp32 or bf16 [groups, beams, vocab] or [groups * beams, vocab], the last
        dimension contiguous; scores fp32 [groups, beams] (-inf: a dead beam); finished
        bool or uint8 [groups, beams] or None; eos the token that finishes a beam (-1: none)."""
        torch = self._torch
        W, V = self.beams, self.vocab
        if logits.dim() == 2 and logits.shape[0] % W == 0:
            logits = logits.unflatten(0, (logits.shape[0] // W, W))
        dt = logits.dtype
        if (logits.dim() != 3 or logits.shape != (logits.shape[0], W, V) or not logits.is_cuda
                or (dt != torch.float32 and dt != torch.bfloat16) or (V > 1 and logits.stride(2) != 1)):
            raise ValueError(f"logits must be a CUDA fp32 or bf16 tensor [groups, {W}, {V}] or [groups * {W}, {V}], "
                             f"contiguous along the vocabulary, got {logits.dtype} {tuple(logits.shape)}")
        G = logits.shape[0]
        _require(scores, (G, W), torch.float32, True, "scores")
        if finished is not None:
            if finished.dtype not in (torch.bool, torch.uint8):
                raise ValueError("finished must be bool or uint8")
            _require(finished, (G, W), finished.dtype, True, "finished")
        _on_current_device(torch, "select", logits, scores, finished)
        tokens, parents, out, done = (_new(torch, scores, None, t, stream)
                                      for t in (torch.int32, torch.int32, torch.float32, torch.bool))
        _check(lib.ling_moe_beam_select(
            self.handle, logits.data_ptr(),
            LING_MOE_TYPE_F32 if dt == torch.float32 else LING_MOE_TYPE_BF16, logits.stride(0), logits.stride(1), G, scores.data_ptr(), finished.data_ptr() if finished is not None else None, int(eos),
            tokens.data_ptr(), parents.data_ptr(), out.data_ptr(), done.data_ptr(), _raw_stream(torch, stream)))
        return tokens, parents, out, done

    def reorder(self, states, parents, slots=None, stream=None):
        """In every tensor of `states` (contiguous, [rows, ...]; one tensor or a list of them, all
        with the same number of rows) the row of beam (g, w) becomes the row that beam
        (g, parents[g, w]) had; in place.  parents: int32 [groups, beams]; slots: the beams'
        rows, int32 [groups, beams] (None: row g * beams + w)."""
        torch = self._torch
        states = [states] if torch.is_tensor(states) else list(states)
        if parents.dim() != 2:
            raise ValueError("parents must be 2-D [groups, beams]")
        G = parents.shape[0]
        _require(parents, (G, self.beams), torch.int32, True, "parents")
        if slots is not None:
            _require(slots, (G, self.beams), torch.int32, True, "slots")
        _on_current_device(torch, "reorder", parents, slots, *states)
        if not states:
            return
        rows = states[0].shape[0] if states[0].dim() else 0
        for t in states:
            if t.dim() < 1 or t.shape[0] != rows or not t.is_contiguous():
                raise ValueError("states must be contiguous CUDA tensors with the same number of rows")
        n = len(states)
        ptr = (ctypes.c_void_p * n)(*[t.data_ptr() for t in states])
        nb = (ctypes.c_size_t * n)(*[(t.numel() // rows if rows else 0) * t.element_size() for t in states])
        _check(lib.ling_moe_beam_reorder(ptr, nb, n, rows, slots.data_ptr() if slots is not None else None,
                                         parents.data_ptr(), G, self.beams, _raw_stream(torch, stream)))

    def launch_count(self) -> int:
        return lib.ling_moe_beam_launch_count(self.handle)


class BlockFP8Linear(_Handle):
    """y = x W^T with e4m3 weights that carry one fp32 scale per 128 x 128 block.

    codes: [out_features, in_features], torch.float8_e4m3fn or its bytes as uint8;
    scales: fp32 [ceil(out / 128), ceil(in / 128)]; contiguous CUDA tensors, copied.
    Tokens are bf16 and are quantised per call (one scale per token and 128 inputs).
    The arithmetic is defined at ling_moe_fp8_linear_forward in ling_moe.h."""

    _destroy = "ling_moe_fp8_linear_destroy"

    def __init__(self, codes, scales, max_tokens: int):
        import torch  # device memory and streams only
        if codes.dim() != 2 or codes.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise ValueError("codes must be 2-D float8_e4m3fn or uint8")
        self.out_features, self.in_features = codes.shape
        self.max_tokens = int(max_tokens)
        _require(codes, tuple(codes.shape), codes.dtype, True, "codes")
        _require(scales, (-(-codes.shape[0] // 128), -(-codes.shape[1] // 128)), torch.float32, True, "scales")
        _on_current_device(torch, "BlockFP8Linear", codes, scales)
        h = ctypes.c_void_p()
        _check(lib.ling_moe_fp8_linear_create(codes.data_ptr(), scales.data_ptr(), self.out_features,
                                              self.in_features, self.max_tokens, ctypes.byref(h)))
        self.handle = h.value
        self._torch = torch

    def forward(self, x, out=None, out_dtype=None, stream=None):
        """[T, out_features] of x [T, in_features] (bf16; rows may be strided).  out_dtype: bf16
        (default) or fp32; out: a tensor to write, rows may be strided."""
        torch = self._torch
        N, K = self.out_features, self.in_features
        T = x.shape[0] if x.dim() == 2 else -1
        if x.shape != (T, K) or x.dtype != torch.bfloat16 or not x.is_cuda or (K > 1 and x.stride(1) != 1):
            raise ValueError(f"x must be a CUDA bf16 tensor [T, {K}] with contiguous rows, got {x.dtype} "
                             f"{tuple(x.shape)} on {x.device}")
        bf16 = (out_dtype if out is None else out.dtype) in (None, torch.bfloat16)
        if out is None and out_dtype in (None, torch.bfloat16, torch.float32):
            out = _new(torch, x, (T, N), torch.bfloat16 if bf16 else torch.float32, stream)
        elif (out is None or out.shape != (T, N) or out.dtype not in (torch.bfloat16, torch.float32)
              or out.dtype != (out_dtype or out.dtype) or not out.is_cuda or (N > 1 and out.stride(1) != 1)):
            raise ValueError(f"out must be a CUDA bf16 or fp32 tensor [{T}, {N}] with contiguous rows, got "
                             + (f"{out.dtype} {tuple(out.shape)} on {out.device}" if out is not None else f"{out_dtype}"))
        _on_current_device(torch, "forward", x, out)
        _check(lib.ling_moe_fp8_linear_forward(
            self.handle, x.data_ptr(), x.stride(0), T, out.data_ptr(), LING_MOE_TYPE_BF16 if bf16 else LING_MOE_TYPE_F32,
            out.stride(0), _raw_stream(torch, stream)))
        return out

    __call__ = forward

    def status(self, stream=None) -> int:
        """Status code of the handle's device work (does not raise on DEVICE_TIMEOUT)."""
        return lib.ling_moe_fp8_linear_status(self.handle, _raw_stream(self._torch, stream))

    def launch_count(self) -> int:
        return lib.ling_moe_fp8_linear_launch_count(self.handle)

    def test_set_wait(self, skip_cta: int, wait_limit_ns: int = 0):
        """Test hook (see ling_moe_fp8_linear_test_set_wait)."""
        _check(lib.ling_moe_fp8_linear_test_set_wait(self.handle, skip_cta, wait_limit_ns))


class GatedDeltaRule(_Handle):
    """The gated delta rule of the linear-attention layers (definition: ling_moe.h).

    Per value head a fp32 state [head_k, head_v] in a pool [slots, v_heads, head_k, head_v]
    that `step` (decode and verify windows) and `prefill` (packed prompts) update in place.
    q and k are normalised inside; g are log-decays (<= 0), per channel [..., v_heads, head_k]
    or per head [..., v_heads]; beta are the write strengths.  scale: of the output
    (None: head_k ** -0.5).  max_tokens: of a prefill call, which sizes its workspace (1
    for a handle that only steps); max_seqs: of any call."""

    _destroy = "ling_moe_delta_destroy"
    MAX_STEP = 8

    def __init__(self, k_heads: int, v_heads: int, head_k: int, head_v: int, max_tokens: int, max_seqs: int,
                 scale: float | None = None):
        import torch  # device memory and streams only
        self.k_heads, self.v_heads, self.head_k, self.head_v = int(k_heads), int(v_heads), int(head_k), int(head_v)
        self.max_tokens, self.max_seqs = int(max_tokens), int(max_seqs)
        if scale is not None and float(scale) == 0.0:
            raise ValueError("scale must not be 0")
        cfg = ling_moe_delta_config_t(self.k_heads, self.v_heads, self.head_k, self.head_v, self.max_tokens,
                                      self.max_seqs, 0.0 if scale is None else float(scale))
        h = ctypes.c_void_p()
        _check(lib.ling_moe_delta_create(ctypes.byref(cfg), ctypes.byref(h)))
        self.handle = h.value
        self._torch = torch

    # ling_moe_delta_io_t: pointers of q, k, v, g, beta; their strides; g's channel stride; out, state; slots
    _pack = struct.Struct("@5P15qqPPiP").pack

    def _io(self, lead, q, k, v, g, beta, state, slots, seqs, out, stream):
        """Check the tensors of a call with leading dimensions `lead` (a tuple); its ling_moe_delta_io_t as bytes, and out."""
        torch = self._torch
        Hk, Hv, dk, dv = self.k_heads, self.v_heads, self.head_k, self.head_v
        nl = len(lead)
        gc = g.dim() == nl + 2
        dev = torch.cuda.current_device() if q.is_cuda else -2
        bf16, f32 = torch.bfloat16, torch.float32
        qk, vh, bh = (*lead, Hk, dk), (*lead, Hv, dv), (*lead, Hv)
        gh = (*lead, Hv, dk) if gc else bh
        if not (q.shape == qk and k.shape == qk and v.shape == vh and g.shape == gh and beta.shape == bh
                and q.dtype == bf16 and k.dtype == bf16 and v.dtype == bf16 and g.dtype == f32 and beta.dtype == f32
                and q.get_device() == dev and k.get_device() == dev and v.get_device() == dev and g.get_device() == dev
                and beta.get_device() == dev):
            for name, t, shape, dt in (("q", q, qk, bf16), ("k", k, qk, bf16), ("v", v, vh, bf16), ("g", g, gh, f32),
                                       ("beta", beta, bh, f32)):
                if t.shape != shape or t.dtype != dt or t.get_device() != dev:
                    raise ValueError(f"{name} must be a CUDA {dt} tensor of shape {shape} on the current device, got "
                                     f"{t.dtype} {tuple(t.shape)} on {t.device}")
        sq, sk, sv, sg, sb = q.stride(), k.stride(), v.stride(), g.stride(), beta.stride()
        if sq[-1] != 1 or sk[-1] != 1 or sv[-1] != 1:
            raise ValueError("q, k and v must be contiguous along their last dimension")
        if gc and sg[-1] not in (0, 1):
            raise ValueError("g must be contiguous (or expanded) along its last dimension")
        if (state.shape != (state.shape[0] if state.dim() else 0, Hv, dk, dv) or state.dtype != f32
                or state.get_device() != dev or not state.is_contiguous()):
            raise ValueError(f"state must be a contiguous CUDA float32 tensor [slots, {Hv}, {dk}, {dv}] on the current "
                             f"device, got {state.dtype} {tuple(state.shape)} on {state.device}")
        if slots is not None:
            _require(slots, (seqs,), torch.int32, True, "slots")
        if out is None:
            out = _new(torch, q, vh, bf16, stream)
        else:
            _require(out, vh, bf16, True, "out")
        if slots is not None or out.get_device() != dev:
            _on_current_device(torch, "delta rule", slots, out)
        if nl == 1:  # no dimension of sequences
            sq, sk, sv, sg, sb = (0, *sq), (0, *sk), (0, *sv), (0, *sg), (0, *sb)
        io = self._pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), *sq[:3], *sk[:3], *sv[:3],
                        *sg[:3], *sb, sg[3] if gc else 0, out.data_ptr(), state.data_ptr(), state.shape[0],
                        slots.data_ptr() if slots is not None else 0)
        return io, out

    def step(self, q, k, v, g, beta, state, slots=None, accepted=None, out=None, stream=None):
        """out bf16 [B, n, v_heads, head_v] of the next n (<= 8) tokens of B sequences: q, k
        [B, n, k_heads, head_k], v [B, n, v_heads, head_v], g, beta [B, n, v_heads(, head_k)].
        slots: int32 [B], the sequences' rows of `state` (None: 0..B-1; outside the pool: padding,
        left untouched); accepted: int32 [B], how many tokens each state advances by (None: all)."""
        torch = self._torch
        if q.dim() != 4:
            raise ValueError("q must be 4-D [sequences, tokens, heads, head_k]")
        B, n = q.shape[0], q.shape[1]
        io, out = self._io((B, n), q, k, v, g, beta, state, slots, B, out, stream)
        if accepted is not None:
            _require(accepted, (B,), torch.int32, True, "accepted")
            _on_current_device(torch, "step", accepted)
        _check(lib.ling_moe_delta_step(self.handle, io, B, n,
                                       accepted.data_ptr() if accepted is not None else None,
                                       _raw_stream(torch, stream)))
        return out

    def prefill(self, q, k, v, g, beta, state, cu_seqlens, slots=None, fresh=None, out=None, stream=None):
        """out bf16 [T, v_heads, head_v] of packed sequences: tokens cu_seqlens[i] .. cu_seqlens[i + 1]
        (int32 [S + 1], on the GPU) are sequence i.  fresh: bool or uint8 [S], sequences that start
        from a zero state (None: all start from their slot's)."""
        torch = self._torch
        if q.dim() != 3:
            raise ValueError("q must be 3-D [tokens, heads, head_k]")
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            raise ValueError("cu_seqlens must be 1-D [sequences + 1]")
        S = cu_seqlens.shape[0] - 1
        _require(cu_seqlens, (S + 1,), torch.int32, True, "cu_seqlens")
        if fresh is not None:
            if fresh.dtype not in (torch.bool, torch.uint8):
                raise ValueError("fresh must be bool or uint8")
            _require(fresh, (S,), fresh.dtype, True, "fresh")
        io, out = self._io((q.shape[0],), q, k, v, g, beta, state, slots, S, out, stream)
        _on_current_device(torch, "prefill", cu_seqlens, fresh)
        _check(lib.ling_moe_delta_prefill(self.handle, io, q.shape[0], cu_seqlens.data_ptr(), S,
                                          fresh.data_ptr() if fresh is not None else None,
                                          _raw_stream(torch, stream)))
        return out

    def status(self, stream=None) -> int:
        """Status code of the handle's device work (does not raise on DEVICE_TIMEOUT)."""
        return lib.ling_moe_delta_status(self.handle, _raw_stream(self._torch, stream))

    def launch_count(self) -> int:
        return lib.ling_moe_delta_launch_count(self.handle)

    def test_set_wait(self, skip: bool, wait_limit_ns: int = 0):
        """Test hook (see ling_moe_delta_test_set_wait)."""
        _check(lib.ling_moe_delta_test_set_wait(self.handle, int(skip), wait_limit_ns))
