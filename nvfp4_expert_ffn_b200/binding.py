"""Thin Python binding of libmoe_nvfp4.so (argument marshalling only).

Every function here has the name of the C entry point it calls (include/moe_nvfp4.h) and
takes torch tensors that already live on the GPU; it passes their device pointers, sizes
and the current CUDA stream through ctypes and raises ``MoeError`` on a non-zero status.
No computation happens here: when the shared library is missing, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# MOE_NVFP4_LIB selects another build of the same library (e.g. the timeline-trace build)
LIB_PATH = os.environ.get("MOE_NVFP4_LIB") or os.path.join(_PKG, "lib", "libmoe_nvfp4.so")

MOE_OK = 0
MOE_FFN_ACCUMULATE, MOE_FFN_PER_ASSIGN = 0, 1
MOE_PATH_AUTO, MOE_PATH_DECODE, MOE_PATH_PREFILL, MOE_PATH_CUDA_CORE = 0, 1, 2, 3
MOE_OP_LAYER, MOE_OP_ROUTE, MOE_OP_QUANT, MOE_OP_FFN, MOE_OP_LAYER_DECODE = 0, 1, 2, 3, 4
MOE_OP_FFN_STATIC = 5
MOE_ERR_INVALID_ARG, MOE_ERR_TIMEOUT, MOE_ERR_WORKSPACE = 1, 4, 5
MOE_TYPE_BF16, MOE_TYPE_F32 = 0, 1
DEFAULT_WAIT_LIMIT_NS = 2_000_000_000

# (name, restype, argtypes) of every C export; tests check the header declares the same set
_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
EXPORTS = {
    "nvfp4_quantize_act": (_I32, [_P, _I64, _I32, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_route": (_I32, [_P, _I32, _I32, _P, _P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_permute": (_I32, [_P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_route_noalloc": (_I32, [_P, _I32, _I32, _P, _P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "moe_pack_experts": (_I32, [_P, _P, _P, _P, _P]),
    "moe_expert_ffn": (_I32, [_P, _P, _P, _I32, _P, _I32, _P, _P, _P, _I32, _I32, _P, _P, _P,
                              _SZ, _P]),
    "moe_expert_ffn_static": (_I32, [_P, _I32, _P, _P, _P, _I32, _P, _P, _P, _I32, _P, _P, _P, _SZ, _P]),
    "moe_combine": (_I32, [_I32, _I32, _I32, _I32, _P, _P, _P, _P, _I32, _P, _P]),
    "moe_expert_hist": (_I32, [_P, _I32, _P, _P, _I32, _P]),
    "moe_layer_decode": (_I32, [_P, _I32, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                _P, _P, _I32, _P, _SZ, _P]),
    "moe_qk_norm_rope": (_I32, [_P, _I64, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P]),
    "nvfp4_kv_append": (_I32, [_P, _I64, _P, _I64, _P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P]),
    "nvfp4_kv_read": (_I32, [_P, _P, _I64, _I32, _P, _P, _P]),
    "nvfp4_kv_attention": (_I32, [_P, _I64, _I32, _I32, _P, _P, _P, _I32, _I32, _I32, _P, ctypes.c_float,
                                  _I32, _P, _P, _P, _SZ, _P]),
    "nvfp4_kv_attention_workspace": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32]),
    "moe_workspace_size": (_SZ, [_I32, _I64, _I32, _I32, _I32, _I32]),
    "moe_get_device_status": (_I32, [_P, _I32, ctypes.POINTER(_I32)]),
    "moe_set_wait_limit_ns": (_I32, [ctypes.c_uint64]),
    "moe_hot_tier_update": (_I32, [_P, _P, _I32, _P, _P, _P]),
    "moe_set_l2_persisting": (_I32, [_SZ, ctypes.POINTER(_SZ)]),
    "moe_status_string": (ctypes.c_char_p, [_I32]),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_version": (_I32, []),
    "moe_launch_count": (ctypes.c_uint64, []),
}


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str):
        super().__init__(f"{fn} failed with status {status}: {detail}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load the shared library once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m nvfp4_expert_ffn_b200.build` (no CPU fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, status: int):
    if status != MOE_OK:
        L = lib()
        raise MoeError(fn, status, L.moe_last_error().decode() or
                       L.moe_status_string(status).decode())


# ------------------------------------------------------------------------- weights

class _WeightsC(ctypes.Structure):
    _fields_ = [("E", _I32), ("d", _I32), ("I", _I32),
                ("gu_codes", _P), ("gu_scales", _P), ("gu_ts", _P),
                ("dn_codes", _P), ("dn_scales", _P), ("dn_ts", _P),
                ("gu_sf_tiled", _P), ("dn_sf_tiled", _P),
                ("dec_pack", _P), ("hot_pack", _P), ("hot_slot", _P), ("n_hot", _I32)]


class _ExpertsC(ctypes.Structure):
    _fields_ = [("routed", _WeightsC), ("shared", _WeightsC), ("has_shared", _I32)]


@dataclass
class ExpertWeights:
    """NVFP4 weights of an expert group on the GPU (natural layout, see moe_nvfp4.h)."""
    gu_codes: Optional[torch.Tensor]   # uint8 [E][2I][d/2]
    gu_scales: Optional[torch.Tensor]  # uint8 [E][2I][d/16]
    gu_ts: torch.Tensor                # float32 [E][2]
    dn_codes: Optional[torch.Tensor]   # uint8 [E][d][I/2]
    dn_scales: Optional[torch.Tensor]  # uint8 [E][d][I/16]
    dn_ts: torch.Tensor                # float32 [E]
    gu_sf_tiled: Optional[torch.Tensor] = None
    dn_sf_tiled: Optional[torch.Tensor] = None
    dec_pack: Optional[torch.Tensor] = None
    dims: tuple = ()                   # (E, d, I), taken from gu_codes when not given
    hot_pack: Optional[torch.Tensor] = None   # uint8: n_hot experts' decode-pack units
    hot_slot: Optional[torch.Tensor] = None   # int32 [E]: slot in hot_pack or -1
    n_hot: int = 0

    def __post_init__(self):
        if not self.dims:
            E, twoI, dh = self.gu_codes.shape
            self.dims = (E, 2 * dh, twoI // 2)

    @property
    def E(self):
        return self.dims[0]

    @property
    def d(self):
        return self.dims[1]

    @property
    def I(self):
        return self.dims[2]

    def release_natural(self) -> None:
        """Drop the natural-layout arrays and the re-tiled scales, keeping the decode pack and
        the tensor scales: enough for moe_layer_decode and the DECODE path, with every
        weight byte held once."""
        if self.dec_pack is None:
            raise ValueError("release_natural needs the decode pack (moe_pack_experts)")
        self.gu_codes = self.gu_scales = self.dn_codes = self.dn_scales = None
        self.gu_sf_tiled = self.dn_sf_tiled = None

    def struct(self) -> _WeightsC:
        p = lambda t: None if t is None else _ptr(t).value  # noqa: E731
        return _WeightsC(self.E, self.d, self.I, p(self.gu_codes), p(self.gu_scales),
                         p(self.gu_ts), p(self.dn_codes), p(self.dn_scales), p(self.dn_ts),
                         p(self.gu_sf_tiled), p(self.dn_sf_tiled), p(self.dec_pack),
                         p(self.hot_pack), p(self.hot_slot), self.n_hot)


@dataclass
class Experts:
    routed: ExpertWeights
    shared: Optional[ExpertWeights] = None
    _c: Optional[_ExpertsC] = field(default=None, repr=False)

    def struct(self) -> _ExpertsC:
        sh = self.shared.struct() if self.shared is not None else _WeightsC()
        self._c = _ExpertsC(self.routed.struct(), sh, 1 if self.shared is not None else 0)
        return self._c


# ------------------------------------------------------------------------- calls

def moe_workspace_size(op: int, T: int, d: int, E: int, k: int, I: int) -> int:
    return int(lib().moe_workspace_size(op, T, d, E, k, I))


def nvfp4_quantize_act(x, codes, scales, ts_out, ts_in=None, ws=None, stream=None):
    rows, cols = x.shape
    _check("nvfp4_quantize_act", lib().nvfp4_quantize_act(
        _ptr(x), rows, cols, _ptr(ts_in), _ptr(codes), _ptr(scales), _ptr(ts_out), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def moe_route(x, Wr, br, k, topk_idx, topk_w, counts, offsets, sorted_assign, assign_pos,
              ws, stream=None):
    T, d = x.shape
    E = Wr.shape[0]
    _check("moe_route", lib().moe_route(
        _ptr(x), T, d, _ptr(Wr), _ptr(br), E, k, _ptr(topk_idx), _ptr(topk_w), _ptr(counts),
        _ptr(offsets), _ptr(sorted_assign), _ptr(assign_pos), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def moe_layer_decode(x, ts_in, Wr, br, experts: "Experts", k, xq_codes, xq_scales, xq_ts, topk_idx,
                     topk_w, counts, offsets, sorted_assign, assign_pos, y_acc, y, rms_renorm, ws,
                     stream=None):
    """The whole layer for at most 8 tokens in one kernel (see include/moe_nvfp4.h); ws must
    be zero-filled before its first use."""
    T = x.shape[0]
    s = experts.struct()
    _check("moe_layer_decode", lib().moe_layer_decode(
        _ptr(x), T, _ptr(ts_in), _ptr(Wr), _ptr(br), ctypes.byref(s), k, _ptr(xq_codes),
        _ptr(xq_scales), _ptr(xq_ts), _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(offsets),
        _ptr(sorted_assign), _ptr(assign_pos), _ptr(y_acc), _ptr(y), 1 if rms_renorm else 0,
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_route_noalloc(x, Wr, br, k, topk_idx, topk_w, counts, offsets, sorted_assign, assign_pos,
                      stream=None):
    """moe_route without a workspace: the library uses its own fixed 256 KiB scratch array
    (for callers that cannot allocate device memory; see include/moe_nvfp4.h)."""
    T, d = x.shape
    E = Wr.shape[0]
    _check("moe_route_noalloc", lib().moe_route_noalloc(
        _ptr(x), T, d, _ptr(Wr), _ptr(br), E, k, _ptr(topk_idx), _ptr(topk_w), _ptr(counts),
        _ptr(offsets), _ptr(sorted_assign), _ptr(assign_pos), _stream(stream)))


def moe_permute(topk_idx, E, counts, offsets, sorted_assign, assign_pos, ws, stream=None):
    T, k = topk_idx.shape
    _check("moe_permute", lib().moe_permute(
        _ptr(topk_idx), T, k, E, _ptr(counts), _ptr(offsets), _ptr(sorted_assign),
        _ptr(assign_pos), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_pack_experts(w: ExpertWeights, stream=None, decode_pack: bool = True):
    """Allocate and fill the derived layouts used by the tensor-core paths: re-tiled scales,
    and (decode_pack=True, d % 512 == 0) the decode pack: all weights again as the 18 KB blocks
    the decode kernel copies into shared memory."""
    if w.gu_sf_tiled is None:
        w.gu_sf_tiled = torch.empty_like(w.gu_scales)
    if w.dn_sf_tiled is None:
        w.dn_sf_tiled = torch.empty_like(w.dn_scales)
    if decode_pack and w.dec_pack is None and w.d % 512 == 0:
        w.dec_pack = torch.empty(dec_pack_bytes(w.E, w.d, w.I), dtype=torch.uint8,
                                 device=w.gu_codes.device)
    s = w.struct()
    _check("moe_pack_experts", lib().moe_pack_experts(
        ctypes.byref(s), _ptr(w.gu_sf_tiled), _ptr(w.dn_sf_tiled), _ptr(w.dec_pack),
        _stream(stream)))


def dec_pack_bytes(E: int, d: int, I: int) -> int:
    """Bytes of the decode pack of an expert group (d % 512 == 0, I % 64 == 0)."""
    return E * (I // 64) * (d // 256 + d // 512) * 18432


def moe_expert_ffn(xq_codes, xq_scales, xq_ts, experts: Experts, k, offsets, sorted_assign,
                   topk_w, mode, path, out, shared_out, ws, stream=None):
    T = xq_codes.shape[0]
    s = experts.struct()
    _check("moe_expert_ffn", lib().moe_expert_ffn(
        _ptr(xq_codes), _ptr(xq_scales), _ptr(xq_ts), T, ctypes.byref(s), k, _ptr(offsets),
        _ptr(sorted_assign), _ptr(topk_w), mode, path, _ptr(out), _ptr(shared_out), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def moe_expert_ffn_static(x, experts: Experts, in_scale_gu, in_scale_dn, k, offsets, sorted_assign,
                          topk_w, mode, out, shared_out, ws, stream=None):
    T = x.shape[0]
    s = experts.struct()
    _check("moe_expert_ffn_static", lib().moe_expert_ffn_static(
        _ptr(x), T, ctypes.byref(s), _ptr(in_scale_gu), _ptr(in_scale_dn), k, _ptr(offsets),
        _ptr(sorted_assign), _ptr(topk_w), mode, _ptr(out), _ptr(shared_out), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def moe_combine(T, d, k, mode, expert_out, shared_out, topk_w, assign_pos, rms_renorm, y,
                stream=None):
    _check("moe_combine", lib().moe_combine(
        T, d, k, mode, _ptr(expert_out), _ptr(shared_out), _ptr(topk_w), _ptr(assign_pos),
        1 if rms_renorm else 0, _ptr(y), _stream(stream)))


def moe_expert_hist(counts, cum, rank_out=None, reset=False, stream=None):
    _check("moe_expert_hist", lib().moe_expert_hist(
        _ptr(counts), counts.numel(), _ptr(cum), _ptr(rank_out), 1 if reset else 0,
        _stream(stream)))


def moe_launch_count() -> int:
    """Kernels this library has enqueued in this process (graph replays not counted)."""
    return int(lib().moe_launch_count())


def moe_get_device_status(clear=True, stream=None) -> int:
    out = _I32(0)
    _check("moe_get_device_status", lib().moe_get_device_status(_stream(stream),
                                                                 1 if clear else 0,
                                                                 ctypes.byref(out)))
    return out.value


def moe_hot_tier_update(w: ExpertWeights, rank, n_hot: int, stream=None) -> None:
    """Copy the units of experts rank[:n_hot] into w's hot tier (allocated here on first
    use, sized for n_hot) and point w at it; n_hot = 0 turns the tier off."""
    if n_hot > 0 and (w.hot_pack is None or w.hot_pack.numel() < dec_pack_bytes(n_hot, w.d, w.I)):
        w.hot_pack = torch.empty(dec_pack_bytes(n_hot, w.d, w.I), dtype=torch.uint8,
                                 device=w.dec_pack.device)
    if w.hot_slot is None:
        w.hot_slot = torch.empty(w.E, dtype=torch.int32, device=w.dec_pack.device)
    s = w.struct()
    _check("moe_hot_tier_update", lib().moe_hot_tier_update(
        ctypes.byref(s), _ptr(rank), n_hot, _ptr(w.hot_pack), _ptr(w.hot_slot), _stream(stream)))
    w.n_hot = n_hot


def moe_set_l2_persisting(nbytes: int) -> int:
    """Set this process's L2 set-aside for persisting lines (clamped to the device's
    maximum; 0 releases it); returns the size in effect."""
    out = _SZ(0)
    _check("moe_set_l2_persisting", lib().moe_set_l2_persisting(int(nbytes), ctypes.byref(out)))
    return int(out.value)


def moe_set_wait_limit_ns(ns: int) -> None:
    _check("moe_set_wait_limit_ns", lib().moe_set_wait_limit_ns(int(ns)))


# ------------------------------------------------------------------------- key/value cache

class _CacheC(ctypes.Structure):
    _fields_ = [("n_pages", _I32), ("page_size", _I32), ("Hkv", _I32), ("D", _I32), ("k_codes", _P),
                ("k_scales", _P), ("v_codes", _P), ("v_scales", _P), ("k_ts", _P), ("v_ts", _P)]


class _PrepC(ctypes.Structure):
    _fields_ = [("q_weight", _P), ("k_weight", _P), ("eps", ctypes.c_double), ("inv_freq", _P),
                ("rot_dim", _I32), ("interleaved", _I32), ("rot_scale", ctypes.c_double)]


def _need(t: Optional[torch.Tensor], name: str, dtype, shape, dev: int) -> Optional[int]:
    """The device pointer of a contiguous tensor of this type and shape on GPU `dev` (None in,
    None out). Calls of a few microseconds go through here: plain comparisons only."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on device {dev}, got "
                         f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _head_rows(t: torch.Tensor, name: str, T: int, D: int, dev: int):
    """Pointer, token stride and heads of bf16 rows [T][heads][D] whose heads lie side by side."""
    if t.dim() != 3 or (t.dtype is not torch.bfloat16 and t.dtype is not torch.int16) or t.get_device() != dev:
        raise ValueError(f"{name} must be a bf16 tensor [T][heads][D] on device {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    n, heads, d = t.shape
    s0, s1, s2 = t.stride()
    if n != T or d != D or s2 != 1 or (heads > 1 and s1 != D):
        raise ValueError(f"{name} must be [{T}][heads][{D}] with contiguous heads, got {tuple(t.shape)} "
                         f"with strides {t.stride()}")
    return t.data_ptr(), (s0 if n > 1 else heads * D), heads


def _call(name: str, dev: int, stream, *args) -> None:
    """lib().<name>(*args, stream) with the tensors' device as the current one."""
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev)
    else:
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors are on device {dev}")
        s = stream.cuda_stream
    f = getattr(lib(), name)
    if torch._C._cuda_getDevice() == dev:
        status = f(*args, s)
    else:
        with torch.cuda.device(dev):
            status = f(*args, s)
    if status != MOE_OK:
        _check(name, status)


@dataclass(frozen=True)
class KVCache:
    """A paged NVFP4 key/value cache of one layer (see moe_kv_cache_t in include/moe_nvfp4.h).

    Token slot s is row s % page_size of page s // page_size."""
    k_codes: torch.Tensor   # uint8 [n_pages][Hkv][page_size][D/2]
    k_scales: torch.Tensor  # uint8 [n_pages][Hkv][page_size][D/16]
    v_codes: torch.Tensor
    v_scales: torch.Tensor
    k_ts: Optional[torch.Tensor] = None  # float32 [Hkv]: static tensor scales (None: 1)
    v_ts: Optional[torch.Tensor] = None

    def __post_init__(self):
        if self.k_codes.dim() != 4:
            raise ValueError("k_codes must be [n_pages][Hkv][page_size][D/2]")
        n, H, ps, dh = self.k_codes.shape
        dev, u8 = self.k_codes.get_device(), torch.uint8
        p = [_need(self.k_codes, "k_codes", u8, (n, H, ps, dh), dev),
             _need(self.k_scales, "k_scales", u8, (n, H, ps, dh // 8), dev),
             _need(self.v_codes, "v_codes", u8, (n, H, ps, dh), dev),
             _need(self.v_scales, "v_scales", u8, (n, H, ps, dh // 8), dev),
             _need(self.k_ts, "k_ts", torch.float32, (H,), dev), _need(self.v_ts, "v_ts", torch.float32, (H,), dev)]
        c = _CacheC(n, ps, H, 2 * dh, *p)
        for name, value in (("n_pages", n), ("page_size", ps), ("Hkv", H), ("D", 2 * dh), ("dev", dev), ("_c", c),
                            ("ref", ctypes.byref(c))):
            object.__setattr__(self, name, value)

    @classmethod
    def allocate(cls, n_pages: int, page_size: int, Hkv: int, D: int, k_ts=None, v_ts=None, device="cuda"):
        """An empty cache (all codes and scales zero)."""
        def z(n):
            return torch.zeros(n_pages, Hkv, page_size, n, dtype=torch.uint8, device=device)
        return cls(z(D // 2), z(D // 16), z(D // 2), z(D // 16), k_ts, v_ts)

    @property
    def device(self):
        return self.k_codes.device


@dataclass(frozen=True)
class QKPrep:
    """Norm and rotation of query and key heads (see moe_qk_prep_t): weights None for no norm,
    inv_freq None for no rotation."""
    q_weight: Optional[torch.Tensor] = None  # float32 [D]
    k_weight: Optional[torch.Tensor] = None  # float32 [D]
    eps: float = 1e-6
    inv_freq: Optional[torch.Tensor] = None  # float32 [rot_dim / 2]
    interleaved: bool = False
    rot_scale: float = 1.0

    # C structures by (D, device); each object's own, dataclasses.replace makes an empty one
    _c: dict = field(init=False, default_factory=dict, repr=False, compare=False)

    def ref(self, D: int, dev: int):
        """A reference to the C structure for heads of D on GPU `dev`, built and checked once."""
        r = self._c.get((D, dev))
        if r is None:
            f32 = torch.float32
            half = 0 if self.inv_freq is None else self.inv_freq.numel()
            r = self._c[(D, dev)] = ctypes.byref(_PrepC(
                _need(self.q_weight, "q_weight", f32, (D,), dev), _need(self.k_weight, "k_weight", f32, (D,), dev), self.eps,
                _need(self.inv_freq, "inv_freq", f32, (half,), dev), 2 * half, 1 if self.interleaved else 0, self.rot_scale))
        return r


def moe_qk_norm_rope(q, k, positions, prep: QKPrep, q_out, k_out, stream=None):
    """Norm and rotation of q [T][Hq][D] and k [T][Hkv][D] (either may be None) into contiguous
    outputs; positions int32 [T] (None without a rotation)."""
    x = q if q is not None else k
    if x is None or x.dim() != 3:
        raise ValueError("q or k must be given, as [T][heads][D]")
    T, _, D = x.shape
    dev = x.get_device()
    qp, qs, Hq = (None, 0, 0) if q is None else _head_rows(q, "q", T, D, dev)
    kp, ks, Hkv = (None, 0, 0) if k is None else _head_rows(k, "k", T, D, dev)
    qo = None if q is None else _need(q_out, "q_out", q.dtype, (T, Hq, D), dev)
    ko = None if k is None else _need(k_out, "k_out", k.dtype, (T, Hkv, D), dev)
    pos = _need(positions, "positions", torch.int32, (T,), dev)
    _call("moe_qk_norm_rope", dev, stream, qp, qs, kp, ks, T, Hq, Hkv, D, pos, prep.ref(D, dev), qo, ko)


def nvfp4_kv_append(q, k, v, positions, slots, prep: QKPrep, cache: KVCache, q_out, stream=None):
    """Norm and rotation of q and k, and k and v quantised into the cache at slots int32 [T]; q
    (with q_out) may be None."""
    if k.dim() != 3:
        raise ValueError("k must be [T][Hkv][D]")
    T, D, dev, i32 = k.shape[0], cache.D, cache.dev, torch.int32
    if k.shape != (T, cache.Hkv, D) or v.shape != k.shape:
        raise ValueError(f"k and v must be [T][{cache.Hkv}][{D}], got {tuple(k.shape)} and {tuple(v.shape)}")
    qp, qs, Hq = (None, 0, 0) if q is None else _head_rows(q, "q", T, D, dev)
    kp, ks, _ = _head_rows(k, "k", T, D, dev)
    vp, vs, _ = _head_rows(v, "v", T, D, dev)
    qo = None if q is None else _need(q_out, "q_out", q.dtype, (T, Hq, D), dev)
    pos, sl = _need(positions, "positions", i32, (T,), dev), _need(slots, "slots", i32, (T,), dev)
    _call("nvfp4_kv_append", dev, stream, qp, qs, kp, ks, vp, vs, T, Hq, pos, sl, prep.ref(D, dev), cache.ref, qo)


def nvfp4_kv_read(cache: KVCache, slots, k_out, v_out, stream=None):
    """Cached rows at slots int32 [n] into k_out and v_out [n][Hkv][D] (bf16 or float32, either
    may be None); a negative slot gives zeros."""
    out = k_out if k_out is not None else v_out
    if out is None:
        raise ValueError("k_out or v_out must be given")
    n, dev = slots.numel(), cache.dev
    f32 = out.dtype is torch.float32
    if not f32 and out.dtype is not torch.bfloat16 and out.dtype is not torch.int16:
        raise ValueError("k_out and v_out must be bf16 or float32")
    shape = (n, cache.Hkv, cache.D)
    ko, vo = _need(k_out, "k_out", out.dtype, shape, dev), _need(v_out, "v_out", out.dtype, shape, dev)
    sl = _need(slots, "slots", torch.int32, (n,), dev)
    _call("nvfp4_kv_read", dev, stream, cache.ref, sl, n, MOE_TYPE_F32 if f32 else MOE_TYPE_BF16, ko, vo)


def nvfp4_kv_attention_workspace(T: int, n_seqs: int, max_q: int, Hq: int, cache: KVCache) -> int:
    """Bytes of workspace of nvfp4_kv_attention for calls up to these sizes."""
    return int(lib().nvfp4_kv_attention_workspace(T, n_seqs, max_q, Hq, cache.Hkv, cache.D))


def nvfp4_kv_attention(q, cu_q, ctx_lens, block_table, max_q: int, cache: KVCache, scale: float, causal: bool, out,
                       lse, ws, stream=None):
    """Attention of packed queries q [T][Hq][D] over the cache (see include/moe_nvfp4.h): sequence
    b's queries are rows cu_q[b] .. cu_q[b+1]-1 (at most max_q), its keys the ctx_lens[b] tokens
    of the pages block_table[b]. lse float32 [T][Hq] may be None."""
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q must be [T][Hq][D] and block_table [n_seqs][max_pages]")
    T, Hq, D = q.shape
    if D != cache.D:
        raise ValueError(f"q has heads of {D}, the cache of {cache.D}")
    dev, i32 = cache.dev, torch.int32
    n, pages = block_table.shape
    qp, qs, _ = _head_rows(q, "q", T, D, dev)
    cu, ctx = _need(cu_q, "cu_q", i32, (n + 1,), dev), _need(ctx_lens, "ctx_lens", i32, (n,), dev)
    table = _need(block_table, "block_table", i32, (n, pages), dev)
    o, e = _need(out, "out", q.dtype, (T, Hq, D), dev), _need(lse, "lse", torch.float32, (T, Hq), dev)
    if ws is None or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on device {dev}")
    _call("nvfp4_kv_attention", dev, stream, qp, qs, T, Hq, cu, ctx, table, n, pages, max_q, cache.ref, scale,
          1 if causal else 0, o, e, ws.data_ptr(), ws.numel() * ws.element_size())
