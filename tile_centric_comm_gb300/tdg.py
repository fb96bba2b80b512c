"""Thin ctypes binding of libtdg (include/tdg.h).  Argument marshalling only:
every step of the path runs in the library's CUDA kernels.  PyTorch supplies
device memory and streams.

The library must have been built (``python -m tile_centric_comm_gb300.build``
or ``__graft_entry__.build()``); when it is missing every call raises -- there
is no fallback.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import struct
import threading

from . import build

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libtdg.so")

TDG_OK = 0
TDG_ERR_INVALID = -1
TDG_ERR_CUDA = -2
TDG_ERR_NOMEM = -3
TDG_ERR_TIMEOUT = -4
TDG_ERR_UNSUPPORTED = -5
TDG_ERR_DEVICE = -6

MODE_SM, MODE_CE, MODE_LL, MODE_SERIAL = 0, 1, 2, 3
MODES = {"sm": MODE_SM, "ce": MODE_CE, "ll": MODE_LL, "serial": MODE_SERIAL}
B_KN, B_NK = 0, 1
MOE_ROUTE, MOE_DISPATCH, MOE_COMBINE, MOE_ALL = 1, 2, 4, 7
KV_BF16, KV_E4M3 = 0, 1
WHERE = {1: "ag_flag", 2: "pipe", 3: "ll", 4: "moe_expert", 5: "ring", 6: "rs_signal",
         7: "page", 8: "pos", 9: "cu", 10: "part", 11: "slot"}
QUANT_ROWS, QUANT_GATED, QUANT_BLOCKS = 0, 1, 2

# every symbol include/tdg.h declares
EXPORTS = [
    "tdg_symm_bytes", "tdg_symm_alloc", "tdg_symm_free", "tdg_symm_region", "tdg_symm_at",
    "tdg_symm_flags", "tdg_symm_counters", "tdg_symm_epoch", "tdg_status", "tdg_strerror",
    "tdg_device_info", "tdg_ag_gemm", "tdg_ag_gemm_all_ranks", "tdg_gemm_rs_stage_bytes", "tdg_gemm_rs",
    "tdg_moe_workspace_bytes", "tdg_moe_dispatch_combine", "tdg_moe_dispatch_combine_noalloc",
    "tdg_allreduce_recv_bytes", "tdg_allreduce", "tdg_flash_decode_part_bytes", "tdg_flash_decode",
    "tdg_paged_pool_bytes", "tdg_rope_append", "tdg_prompt_attention",
    "tdg_paged_decode_part_bytes", "tdg_paged_decode",
    "tdg_quantise", "tdg_scaled_gemm", "tdg_moe_dispatch_e4m3", "tdg_moe_combine_grad", "tdg_moe_dispatch_grad",
]
MOE_STATIC_WORKSPACE_BYTES = 2 * 1024 * 1024

_i32, _i64, _u32, _u64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64
_sz, _vp = ctypes.c_size_t, ctypes.c_void_p


class TdgFault(ctypes.Structure):
    _fields_ = [("code", _i32), ("where", _u32), ("index", _u32), ("epoch", _u32)]


class AgGemmArgs(ctypes.Structure):
    _fields_ = [("world", ctypes.c_int), ("rank", ctypes.c_int), ("Ms", _i64), ("K", _i64),
                ("N", _i64), ("a_off", _sz), ("g_off", _sz), ("B", _vp), ("C", _vp),
                ("b_layout", ctypes.c_int), ("mode", ctypes.c_int), ("producers", ctypes.c_int),
                ("signal_rows", _i64), ("swizzle", ctypes.c_int), ("timeout_ns", _u64),
                ("ll_off", _sz), ("test_skip_notify", _u64), ("source_order", ctypes.c_int),
                ("c_f32", ctypes.c_int), ("cluster", ctypes.c_int), ("stages", ctypes.c_int),
                ("split_tail", ctypes.c_int), ("producer_items", ctypes.c_int),
                ("producer_warps", ctypes.c_int), ("producer_chunk", ctypes.c_int),
                ("push", ctypes.c_int)]


class AgGemmAllArgs(ctypes.Structure):
    _fields_ = [("world", ctypes.c_int), ("Ms", _i64), ("K", _i64), ("N", _i64), ("a_off", _sz),
                ("g_off", _sz), ("b_off", _sz), ("c_off", _sz), ("b_layout", ctypes.c_int),
                ("mode", ctypes.c_int), ("signal_rows", _i64), ("timeout_ns", _u64),
                ("test_skip_notify", _u64), ("c_f32", ctypes.c_int), ("cluster", ctypes.c_int),
                ("stages", ctypes.c_int), ("push", ctypes.c_int)]


class GemmRsArgs(ctypes.Structure):
    _fields_ = [("world", ctypes.c_int), ("M", _i64), ("K", _i64), ("N", _i64), ("a_off", _sz),
                ("b_off", _sz), ("stage_off", _sz), ("out_off", _sz), ("b_layout", ctypes.c_int),
                ("mode", ctypes.c_int), ("timeout_ns", _u64), ("owner_block", ctypes.c_int),
                ("partial_f32", ctypes.c_int), ("cluster", ctypes.c_int), ("stages", ctypes.c_int),
                ("order", ctypes.c_int), ("red_rows", ctypes.c_int), ("spare", ctypes.c_int)]


class MoeArgs(ctypes.Structure):
    _fields_ = [("world", ctypes.c_int), ("T", _i64), ("H", _i64), ("E", ctypes.c_int),
                ("k", ctypes.c_int), ("x_off", _sz), ("topk_off", _sz), ("gate_off", _sz),
                ("out_off", _sz), ("recv", _vp), ("y", _vp), ("counts", _vp), ("base", _vp),
                ("slot", _vp), ("row_src", _vp), ("row_tok", _vp), ("row_k", _vp),
                ("workspace", _vp), ("workspace_bytes", _sz), ("phases", ctypes.c_int)]


class AllReduceArgs(ctypes.Structure):
    _fields_ = [("world", ctypes.c_int), ("count", _i64), ("x_off", _sz), ("recv_off", _sz),
                ("tile_elems", _i64), ("ctas_per_rank", ctypes.c_int), ("timeout_ns", _u64),
                ("test_skip_signal", _u64)]


class FlashDecodeArgs(ctypes.Structure):
    _fields_ = [("world", ctypes.c_int), ("root", ctypes.c_int), ("B", _i64), ("Hq", _i64),
                ("Hkv", _i64), ("D", _i64), ("S", _i64), ("k_off", _sz), ("v_off", _sz),
                ("part_off", _sz), ("q", _vp), ("out", _vp), ("chunk", _i64),
                ("scale", ctypes.c_float)]


class PagedCacheDesc(ctypes.Structure):
    _fields_ = [("pages", _i64), ("page_size", ctypes.c_int), ("kv_type", ctypes.c_int),
                ("Hkv", _i64), ("D", _i64), ("k_off", _sz), ("v_off", _sz), ("k_scale", _vp),
                ("v_scale", _vp)]


class RopeAppendArgs(ctypes.Structure):
    _fields_ = [("world", ctypes.c_int), ("cache", PagedCacheDesc), ("T", _i64), ("B", _i64),
                ("Hq", _i64), ("q", _vp), ("k", _vp), ("v", _vp), ("q_stride", _i64),
                ("k_stride", _i64), ("v_stride", _i64), ("q_out", _vp), ("k_out", _vp),
                ("q_out_stride", _i64), ("k_out_stride", _i64), ("cos_sin", _vp),
                ("max_pos", _i64), ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("axes", ctypes.c_int), ("sections", ctypes.c_int * 3), ("pos", _vp),
                ("pos_stride", _i64), ("cu", _vp), ("table", _vp), ("table_entries", _i64), ("table_stride", _i64),
                ("lens", _vp)]


class PromptAttentionArgs(ctypes.Structure):
    _fields_ = [("Tq", _i64), ("Tk", _i64), ("B", _i64), ("Hq", _i64), ("Hkv", _i64), ("D", _i64),
                ("q", _vp), ("k", _vp), ("v", _vp), ("q_stride", _i64), ("k_stride", _i64),
                ("v_stride", _i64), ("out", _vp), ("out_stride", _i64), ("lse", _vp),
                ("cu_q", _vp), ("cu_k", _vp), ("causal", ctypes.c_int), ("scale", ctypes.c_float)]


class PagedDecodeArgs(ctypes.Structure):
    _fields_ = [("world", ctypes.c_int), ("root", ctypes.c_int), ("cache", PagedCacheDesc),
                ("B", _i64), ("Hq", _i64), ("q", _vp), ("q_stride", _i64), ("out", _vp),
                ("out_stride", _i64), ("lse", _vp), ("table", _vp), ("table_entries", _i64), ("table_stride", _i64),
                ("lens", _vp), ("part_off", _sz), ("scale", ctypes.c_float)]


class QuantiseArgs(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("rows", _i64), ("K", _i64), ("E", _i64), ("x", _vp), ("x_stride", _i64),
                ("codes", _vp), ("codes_stride", _i64), ("scale", _vp), ("scale_stride", _i64), ("count", _vp)]


class ScaledGemmArgs(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64), ("E", _i64), ("a", _vp), ("a_stride", _i64), ("a_scale", _vp),
                ("a_scale_stride", _i64), ("b", _vp), ("b_scale", _vp), ("out", _vp), ("out_stride", _i64),
                ("out_f32", ctypes.c_int), ("base", _vp)]


class MoeDispatchE4m3Args(ctypes.Structure):
    _fields_ = [("world", ctypes.c_int), ("k", ctypes.c_int), ("T", _i64), ("H", _i64), ("x_off", _sz), ("slot", _vp),
                ("codes", _vp), ("scale", _vp)]


class MoeCombineGradArgs(ctypes.Structure):
    _fields_ = [("world", ctypes.c_int), ("k", ctypes.c_int), ("T", _i64), ("H", _i64), ("gate_off", _sz),
                ("dout_off", _sz), ("dgate_off", _sz), ("slot", _vp), ("y", _vp), ("dy", _vp)]


class MoeDispatchGradArgs(ctypes.Structure):
    _fields_ = [("world", ctypes.c_int), ("k", ctypes.c_int), ("T", _i64), ("H", _i64), ("dx_off", _sz), ("slot", _vp),
                ("drecv", _vp)]


class TdgError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} ({code})")


_lib = None
_lock = threading.Lock()


def lib():
    """Open libtdg.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"libtdg.so not found at {LIB_PATH}: build it with "
                    "`python -m tile_centric_comm_gb300.build` (there is no CPU fallback)")
            L = ctypes.CDLL(LIB_PATH)
            L.tdg_symm_bytes.restype = _sz
            L.tdg_symm_bytes.argtypes = [ctypes.c_int, _sz, _sz]
            L.tdg_symm_alloc.restype = ctypes.c_int
            L.tdg_symm_alloc.argtypes = [_vp, _sz, ctypes.c_int, _sz, _sz, ctypes.POINTER(_vp)]
            L.tdg_symm_free.restype = ctypes.c_int
            L.tdg_symm_free.argtypes = [_vp]
            for n in ("tdg_symm_region", "tdg_symm_flags", "tdg_symm_counters"):
                getattr(L, n).restype = _vp
                getattr(L, n).argtypes = [_vp, ctypes.c_int]
            L.tdg_symm_at.restype = _vp
            L.tdg_symm_at.argtypes = [_vp, _vp, ctypes.c_int]
            L.tdg_symm_epoch.restype = _u32
            L.tdg_symm_epoch.argtypes = [_vp]
            L.tdg_status.restype = ctypes.c_int
            L.tdg_status.argtypes = [_vp, _vp, ctypes.POINTER(TdgFault), ctypes.c_int]
            L.tdg_strerror.restype = ctypes.c_char_p
            L.tdg_strerror.argtypes = [ctypes.c_int]
            L.tdg_device_info.restype = ctypes.c_int
            L.tdg_device_info.argtypes = [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
            L.tdg_ag_gemm.restype = ctypes.c_int
            L.tdg_ag_gemm.argtypes = [_vp, ctypes.POINTER(AgGemmArgs), _vp, _vp]
            L.tdg_ag_gemm_all_ranks.restype = ctypes.c_int
            L.tdg_ag_gemm_all_ranks.argtypes = [_vp, ctypes.POINTER(AgGemmAllArgs), _vp, _vp]
            L.tdg_gemm_rs_stage_bytes.restype = _sz
            L.tdg_gemm_rs_stage_bytes.argtypes = [ctypes.c_int, _i64, _i64]
            L.tdg_gemm_rs.restype = ctypes.c_int
            L.tdg_gemm_rs.argtypes = [_vp, ctypes.POINTER(GemmRsArgs), _vp]
            L.tdg_moe_workspace_bytes.restype = _sz
            L.tdg_moe_workspace_bytes.argtypes = [ctypes.c_int, _i64, ctypes.c_int]
            L.tdg_moe_dispatch_combine.restype = ctypes.c_int
            L.tdg_moe_dispatch_combine.argtypes = [_vp, ctypes.POINTER(MoeArgs), _vp]
            L.tdg_allreduce_recv_bytes.restype = _sz
            L.tdg_allreduce_recv_bytes.argtypes = [ctypes.c_int, _i64]
            L.tdg_allreduce.restype = ctypes.c_int
            L.tdg_allreduce.argtypes = [_vp, ctypes.POINTER(AllReduceArgs), _vp]
            L.tdg_flash_decode_part_bytes.restype = _sz
            L.tdg_flash_decode_part_bytes.argtypes = [ctypes.c_int, _i64, _i64, _i64, _i64, _i64]
            L.tdg_flash_decode.restype = ctypes.c_int
            L.tdg_flash_decode.argtypes = [_vp, ctypes.POINTER(FlashDecodeArgs), _vp]
            L.tdg_paged_pool_bytes.restype = _sz
            L.tdg_paged_pool_bytes.argtypes = [_i64, ctypes.c_int, _i64, _i64, ctypes.c_int]
            L.tdg_rope_append.restype = ctypes.c_int
            L.tdg_rope_append.argtypes = [_vp, ctypes.POINTER(RopeAppendArgs), _vp]
            L.tdg_prompt_attention.restype = ctypes.c_int
            L.tdg_prompt_attention.argtypes = [_vp, ctypes.POINTER(PromptAttentionArgs), _vp]
            L.tdg_paged_decode_part_bytes.restype = _sz
            L.tdg_paged_decode_part_bytes.argtypes = [_i64, _i64, _i64]
            L.tdg_paged_decode.restype = ctypes.c_int
            L.tdg_paged_decode.argtypes = [_vp, ctypes.POINTER(PagedDecodeArgs), _vp]
            for n, args in (("tdg_quantise", QuantiseArgs), ("tdg_scaled_gemm", ScaledGemmArgs),
                            ("tdg_moe_dispatch_e4m3", MoeDispatchE4m3Args), ("tdg_moe_combine_grad", MoeCombineGradArgs),
                            ("tdg_moe_dispatch_grad", MoeDispatchGradArgs)):
                getattr(L, n).restype = ctypes.c_int
                getattr(L, n).argtypes = [_vp, ctypes.POINTER(args), _vp]
            L.tdg_moe_dispatch_combine_noalloc.restype = ctypes.c_int
            L.tdg_moe_dispatch_combine_noalloc.argtypes = [_vp, ctypes.POINTER(MoeArgs), _vp]
            _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().tdg_strerror(code).decode()


def _check(rc, what):
    if rc != TDG_OK:
        raise TdgError(rc, what)


def _tensor(t, name, dtype, numel, device=None):
    """Check a tensor handed to the library as a raw pointer: the library sees
    neither strides nor dtype, so it must be a contiguous CUDA tensor of the
    documented element type holding at least `numel` elements."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous (the library reads it row-major)")
    if t.numel() < numel:
        raise ValueError(f"{name}: holds {t.numel()} elements, needs {numel}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, the heap is on {device}")
    return t.data_ptr()


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return _vp(stream.cuda_stream)


def device_info():
    sms, sup = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().tdg_device_info(ctypes.byref(sms), ctypes.byref(sup)), "tdg_device_info")
    return sms.value, bool(sup.value)


class Symm:
    """A symmetric heap of `world` regions carved from one torch allocation."""

    def __init__(self, world: int, region_bytes: int, signals_per_rank: int = 65536,
                 device=None, buffer=None):
        import torch
        region_bytes = (int(region_bytes) + 1023) // 1024 * 1024
        L = lib()
        nbytes = L.tdg_symm_bytes(world, region_bytes, signals_per_rank)
        if buffer is None:
            buffer = torch.empty(nbytes + 1024, dtype=torch.uint8, device=device or "cuda")
        _tensor(buffer, "buffer", torch.uint8, nbytes + 1024)
        self.buf = buffer
        self.device = buffer.device
        self.base_off = (-buffer.data_ptr()) % 1024
        self.base = buffer.data_ptr() + self.base_off
        self.nbytes = nbytes
        self.world = world
        self.region_bytes = region_bytes
        self.nsig = signals_per_rank
        h = _vp()
        _check(L.tdg_symm_alloc(_vp(self.base), nbytes, world, region_bytes, signals_per_rank,
                                ctypes.byref(h)), "tdg_symm_alloc")
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            lib().tdg_symm_free(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def region_ptr(self, rank: int) -> int:
        return lib().tdg_symm_region(self.h, rank)

    def view(self, rank: int, off: int, shape, dtype):
        """A tensor over region `rank` at byte offset `off`."""
        import torch
        n = 1
        for d in shape:
            n *= int(d)
        esz = torch.empty((), dtype=dtype).element_size()
        if not 0 <= rank < self.world:
            raise ValueError(f"rank {rank} outside [0, {self.world})")
        if off < 0 or off % esz or off + n * esz > self.region_bytes:
            raise ValueError(f"view of {n * esz} bytes at offset {off} does not fit a "
                             f"{self.region_bytes}-byte region with {esz}-byte alignment")
        start = self.base_off + rank * self.region_bytes + off
        return self.buf[start:start + n * esz].view(dtype).view(*shape)

    def flags(self, rank: int, n: int):
        import torch
        if not 0 <= rank < self.world or not 0 <= n <= self.nsig:
            raise ValueError(f"flags({rank}, {n}) outside {self.world} ranks x {self.nsig} words")
        start = lib().tdg_symm_flags(self.h, rank) - self.buf.data_ptr()
        return self.buf[start:start + 4 * n].view(torch.int32)

    def counters(self, rank: int, n: int):
        import torch
        if not 0 <= rank < self.world or not 0 <= n <= self.nsig:
            raise ValueError(f"counters({rank}, {n}) outside {self.world} ranks x {self.nsig} words")
        start = lib().tdg_symm_counters(self.h, rank) - self.buf.data_ptr()
        return self.buf[start:start + 4 * n].view(torch.int32)

    def at(self, ptr: int, rank: int):
        return lib().tdg_symm_at(self.h, _vp(ptr), rank)

    def epoch(self) -> int:
        return lib().tdg_symm_epoch(self.h)

    def status(self, stream=None, clear: bool = True):
        f = TdgFault()
        rc = lib().tdg_status(self.h, _stream(stream), ctypes.byref(f), 1 if clear else 0)
        if rc == TDG_ERR_CUDA:
            raise TdgError(rc, "tdg_status")
        return dict(code=f.code, where=WHERE.get(f.where, f.where), index=f.index, epoch=f.epoch)


def ag_gemm(symm: Symm, rank: int, Ms: int, K: int, N: int, a_off: int, g_off: int, B, C,
            mode="sm", b_layout=B_KN, producers=0, signal_rows=0, swizzle=True,
            timeout_ns=0, ll_off=0, test_skip_notify=0, source_order=0, stream=None,
            side_stream=None, c_f32=False, cluster=0, stages=0, split_tail=False,
            producer_items=0, producer_warps=0, producer_chunk=0, push=False):
    """c_f32: C is float32 (the fp32 accumulator, unrounded) instead of bf16.
    cluster / stages / split_tail / producer_items / producer_warps /
    producer_chunk / push choose the schedule (0 / False: the default for the
    shape); see tdg_ag_gemm_args in include/tdg.h."""
    import torch
    dev = symm.buf.device
    # N == 0 runs the AllGather alone: B and C may then be None
    a = AgGemmArgs(world=symm.world, rank=rank, Ms=Ms, K=K, N=N, a_off=a_off, g_off=g_off,
                   B=None if (N == 0 and B is None) else _tensor(B, "B", torch.bfloat16, K * N, dev),
                   C=None if (N == 0 and C is None) else
                   _tensor(C, "C", torch.float32 if c_f32 else torch.bfloat16, symm.world * Ms * N, dev),
                   b_layout=b_layout, mode=MODES[mode],
                   producers=producers, signal_rows=signal_rows, swizzle=1 if swizzle else 0,
                   timeout_ns=timeout_ns, ll_off=ll_off, test_skip_notify=test_skip_notify,
                   source_order=source_order, c_f32=1 if c_f32 else 0, cluster=cluster,
                   stages=stages, split_tail=1 if split_tail else 0, producer_items=producer_items,
                   producer_warps=producer_warps, producer_chunk=producer_chunk,
                   push=1 if push else 0)
    side = _vp(side_stream.cuda_stream) if side_stream is not None else _vp(None)
    _check(lib().tdg_ag_gemm(symm.h, ctypes.byref(a), _stream(stream), side), "tdg_ag_gemm")


def ag_gemm_all_ranks(symm: Symm, Ms: int, K: int, N: int, a_off: int, g_off: int, b_off: int,
                      c_off: int, mode="ce", b_layout=B_KN, signal_rows=0, timeout_ns=0,
                      test_skip_notify=0, stream=None, side_stream=None, c_f32=False,
                      cluster=0, stages=0, push=False):
    """AllGather+GEMM of every rank in one call: C_r = concat(A_0..A_{W-1}) @ B_r,
    with A_r, the gathered buffers, B_r and C_r all in the heap (offsets).
    c_f32: C_r is float32 (the fp32 accumulator, unrounded) instead of bf16.
    push: the copies go step by step, sender s to destination (s + j) mod W."""
    a = AgGemmAllArgs(world=symm.world, Ms=Ms, K=K, N=N, a_off=a_off, g_off=g_off, b_off=b_off,
                      c_off=c_off, b_layout=b_layout, mode=MODES[mode], signal_rows=signal_rows,
                      timeout_ns=timeout_ns, test_skip_notify=test_skip_notify,
                      c_f32=1 if c_f32 else 0, cluster=cluster, stages=stages,
                      push=1 if push else 0)
    side = _vp(side_stream.cuda_stream) if side_stream is not None else _vp(None)
    _check(lib().tdg_ag_gemm_all_ranks(symm.h, ctypes.byref(a), _stream(stream), side),
           "tdg_ag_gemm_all_ranks")


def gemm_rs_stage_bytes(world: int, M: int, N: int) -> int:
    return lib().tdg_gemm_rs_stage_bytes(world, M, N)


def gemm_rs(symm: Symm, M: int, K: int, N: int, a_off: int, b_off: int, stage_off: int,
            out_off: int, mode="sm", b_layout=B_KN, timeout_ns=0, owner_block=0,
            partial_f32=False, stream=None, cluster=0, stages=0, order=0, red_rows=0, spare=0):
    """partial_f32: push fp32 partials (the staging area must then hold
    2 * gemm_rs_stage_bytes(world, M, N) bytes).  cluster / stages / order /
    red_rows / owner_block / spare choose the schedule (0: the default for the
    shape; spare=n > 0 lets CTA pairs on the SMs that 4-CTA clusters leave
    idle take the last n of the world**2 groups of tiles)."""
    a = GemmRsArgs(world=symm.world, M=M, K=K, N=N, a_off=a_off, b_off=b_off,
                   stage_off=stage_off, out_off=out_off, b_layout=b_layout,
                   mode=MODES[mode], timeout_ns=timeout_ns, owner_block=owner_block,
                   partial_f32=1 if partial_f32 else 0, cluster=cluster, stages=stages,
                   order=order, red_rows=red_rows, spare=spare)
    _check(lib().tdg_gemm_rs(symm.h, ctypes.byref(a), _stream(stream)), "tdg_gemm_rs")


def allreduce_recv_bytes(world: int, count: int) -> int:
    return lib().tdg_allreduce_recv_bytes(world, count)


def allreduce(symm: Symm, count: int, x_off: int, recv_off: int, tile_elems=0, ctas_per_rank=0,
              timeout_ns=0, test_skip_signal=0, stream=None):
    a = AllReduceArgs(world=symm.world, count=count, x_off=x_off, recv_off=recv_off,
                      tile_elems=tile_elems, ctas_per_rank=ctas_per_rank, timeout_ns=timeout_ns,
                      test_skip_signal=test_skip_signal)
    _check(lib().tdg_allreduce(symm.h, ctypes.byref(a), _stream(stream)), "tdg_allreduce")


def flash_decode_part_bytes(world: int, B: int, Hq: int, D: int, S: int, chunk: int = 0) -> int:
    return lib().tdg_flash_decode_part_bytes(world, B, Hq, D, S, chunk)


def flash_decode(symm: Symm, B: int, Hq: int, Hkv: int, D: int, S: int, k_off: int, v_off: int,
                 part_off: int, q, out, root: int = 0, chunk: int = 0, scale: float = 0.0,
                 stream=None):
    import torch
    dev = symm.buf.device
    a = FlashDecodeArgs(world=symm.world, root=root, B=B, Hq=Hq, Hkv=Hkv, D=D, S=S, k_off=k_off,
                        v_off=v_off, part_off=part_off,
                        q=_tensor(q, "q", torch.bfloat16, B * Hq * D, dev),
                        out=_tensor(out, "out", torch.bfloat16, B * Hq * D, dev),
                        chunk=chunk, scale=scale)
    _check(lib().tdg_flash_decode(symm.h, ctypes.byref(a), _stream(stream)), "tdg_flash_decode")


def paged_pool_bytes(pages: int, page_size: int, Hkv: int, D: int, e4m3: bool = False) -> int:
    """Bytes of one pool (keys or values) in one rank's region."""
    return lib().tdg_paged_pool_bytes(pages, page_size, Hkv, D, KV_E4M3 if e4m3 else KV_BF16)


class PagedCache:
    """A paged key-value cache in the heap: `pages` pages of `page_size` tokens
    per rank, key pool at k_off and value pool at v_off of every region, each
    (pages, Hkv, page_size, D) in bf16, or in 8 bits (e4m3=True) with one
    float32 scale per key head for keys and for values.  Page id p is page
    p % pages of rank p // pages."""

    def __init__(self, pages: int, page_size: int, Hkv: int, D: int, k_off: int, v_off: int,
                 e4m3: bool = False, k_scale=None, v_scale=None):
        import torch
        if e4m3 != (k_scale is not None) or e4m3 != (v_scale is not None):
            raise ValueError("k_scale and v_scale belong to an 8-bit cache, and only to one")
        self.pages, self.page_size, self.Hkv, self.D = pages, page_size, Hkv, D
        self.k_off, self.v_off, self.e4m3 = k_off, v_off, e4m3
        self.k_scale, self.v_scale = k_scale, v_scale       # kept alive with the description
        self.desc = PagedCacheDesc(
            pages=pages, page_size=page_size, kv_type=KV_E4M3 if e4m3 else KV_BF16, Hkv=Hkv, D=D,
            k_off=k_off, v_off=v_off,
            k_scale=_tensor(k_scale, "k_scale", torch.float32, Hkv) if e4m3 else None,
            v_scale=_tensor(v_scale, "v_scale", torch.float32, Hkv) if e4m3 else None)
        self.device = k_scale.device if e4m3 else None      # that of the scales; the calls compare it with the heap's
        if e4m3 and v_scale.device != self.device:
            raise ValueError(f"v_scale: on {v_scale.device}, k_scale is on {self.device}")
        # the description's fields as the packed calls take them
        self.packed = (pages, page_size, self.desc.kv_type, Hkv, D, k_off, v_off,
                       self.desc.k_scale or 0, self.desc.v_scale or 0)

    def pools(self, symm: Symm, rank: int):
        """The key and the value pool of one rank, as tensors."""
        import torch
        shape = (self.pages, self.Hkv, self.page_size, self.D)
        kind = torch.float8_e4m3fn if self.e4m3 else torch.bfloat16
        return symm.view(rank, self.k_off, shape, kind), symm.view(rank, self.v_off, shape, kind)


def _other_device(cache, device):
    raise ValueError(f"k_scale and v_scale: on {cache.device}, the heap is on {device}")


_torch = _current_raw_stream = _rows = _table = _flat = _matrix = None


def _attn():
    """torch, and the attention and 8-bit entry points of the library taking
    packed arguments (one struct.pack call costs a fraction of filling a ctypes
    structure field by field, and these calls are short)."""
    global _torch, _current_raw_stream, _rows, _table, _flat, _matrix, _Tensor, _t_bf16, _t_i32, _t_f32, _t_i64, _t_e4m3
    import torch
    L = lib()
    # the native checks where they were built for this torch and this Python,
    # else the same checks in Python (5 us a call more)
    _rows, _table, _flat, _matrix = _checked_rows, _checked_table, _checked_flat, _checked_matrix
    path = build.tensors_path(torch.version.__version__)
    if os.path.exists(path):
        loader = importlib.machinery.ExtensionFileLoader("tdg_tensors", path)
        checks = importlib.util.module_from_spec(importlib.util.spec_from_loader("tdg_tensors", loader))
        loader.exec_module(checks)
        checks.setup(torch.Tensor, _checked_rows, _checked_table, _checked_flat, _checked_matrix)
        _rows, _table, _flat, _matrix = checks.rows, checks.table, checks.flat, checks.matrix
    fast = ctypes.CDLL(LIB_PATH)
    for name in ("tdg_rope_append", "tdg_prompt_attention", "tdg_paged_decode", "tdg_quantise", "tdg_scaled_gemm",
                 "tdg_moe_dispatch_e4m3", "tdg_moe_combine_grad", "tdg_moe_dispatch_grad"):
        f = getattr(fast, name)
        f.restype, f.argtypes = ctypes.c_int, [_vp, ctypes.c_char_p, _vp]
        globals()["_" + name] = f
    _current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _Tensor, _t_bf16, _t_i32, _t_f32 = torch.Tensor, torch.bfloat16, torch.int32, torch.float32
    _t_i64, _t_e4m3 = torch.int64, torch.float8_e4m3fn
    _torch = torch
    return L


_DESC = "qiiqqNNPP"                                          # tdg_paged_cache
_pack_rope = struct.Struct("@i4x" + _DESC + "qqqPPPqqqPPqqPqiiiiiiPqPPqqP").pack
_pack_prompt = struct.Struct("@qqqqqqPPPqqqPqPPPif").pack
_pack_decode = struct.Struct("@ii" + _DESC + "qqPqPqPPqqPNf0q").pack
_pack_quantise = struct.Struct("@i4xqqqPqPqPqP").pack
_pack_scaled = struct.Struct("@qqqqPqPqPPPqi4xP").pack
_pack_dispatch_e4m3 = struct.Struct("@iiqqNPPP").pack
_pack_combine_grad = struct.Struct("@iiqqNNNPPP").pack
_pack_dispatch_grad = struct.Struct("@iiqqNPP").pack


def _raw_stream(stream, device):
    """The stream to run on: the given one, or torch's current one."""
    if stream is not None:
        return stream.cuda_stream
    # without building a Stream object (2 us) where torch offers it
    return _current_raw_stream(device.index) if _current_raw_stream else \
        _torch.cuda.current_stream(device).cuda_stream


# csrc/tdg_tensors.cpp does the same checks for tensors that pass them and calls
# these for those that do not
def _checked_rows(t, name, device):
    """Check rows of heads, (rows, heads, D) in bf16, whose rows may be strided
    (columns of a wider buffer); returns (pointer, row stride in elements, rows,
    heads, D)."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype is not _t_bf16:
        raise TypeError(f"{name}: expected torch.bfloat16, got {t.dtype}")
    stride = t.stride()
    if len(stride) != 3:
        raise ValueError(f"{name}: expected (rows, heads, D), got {tuple(t.shape)}")
    n, heads, D = t.shape
    s0, s1, s2 = stride
    if n <= 1 or not heads:
        s0 = heads * D          # no second row, no stride
        if not n or not heads:
            return t.data_ptr(), s0, n, heads, D
    if (s2 != 1 and D > 1) or (s1 != D and heads > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous, strides {stride}")
    if t.get_device() != device.index:
        raise ValueError(f"{name}: on {t.device}, the heap is on {device}")
    return t.data_ptr(), s0, n, heads, D


def _checked_table(table, name, device):
    """Check a page table (sequences, entries), int32, rows possibly strided;
    returns (pointer, entries, row stride, sequences)."""
    if not isinstance(table, _Tensor) or table.dtype is not _t_i32:
        raise TypeError(f"{name}: expected an int32 tensor")
    stride = table.stride()
    if len(stride) != 2:
        raise ValueError(f"{name}: expected (sequences, entries)")
    n, entries = table.shape
    if entries > 1 and stride[1] != 1:
        raise ValueError(f"{name}: expected (sequences, entries) with contiguous rows")
    if table.get_device() != device.index:
        raise ValueError(f"{name}: on {table.device}, the heap is on {device}")
    return table.data_ptr(), entries, entries if n <= 1 else stride[0], n


def _checked_flat(t, name, dtype, numel, device):
    """_tensor's checks, in the order in which they are cheap."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == device.index and t.is_contiguous() \
            and t.numel() >= numel:
        return t.data_ptr()
    return _tensor(t, name, dtype, numel, device)


def _checked_matrix(t, name, dtype, device):
    """Check a matrix whose rows may be strided; returns (pointer, row stride in
    elements, rows, columns)."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    stride = t.stride()
    if len(stride) != 2:
        raise ValueError(f"{name}: expected (rows, columns), got {tuple(t.shape)}")
    rows, columns = t.shape
    if columns > 1 and stride[1] != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous, strides {stride}")
    if t.get_device() != device.index:
        raise ValueError(f"{name}: on {t.device}, the heap is on {device}")
    return t.data_ptr(), columns if rows <= 1 else stride[0], rows, columns


def rope_append(symm: Symm, cache: PagedCache, q, k, v, q_out, cos_sin, pos, table, lens, cu=None,
                k_out=None, sections=None, interleaved=False, stream=None):
    """Turn the queries q (T, Hq, D) and keys k (T, Hkv, D) of T new tokens by
    their positions into q_out and k_out, and write keys and values v into the
    cache.  cos_sin: (positions, rot_dim) float32, cosines then sines (None: no
    rotation); pos: (T,) or (axes, T) int32 with `sections` pairs per axis;
    table: (B, entries) int32 page ids (None: no cache write); lens: (B,) int32
    lengths with the new tokens; cu: (B + 1,) int32 row offsets (None: one row
    per sequence).  q and q_out may be None, q_out may be q, k_out may be k."""
    if _torch is None:
        _attn()
    dev, i32 = symm.device, _t_i32
    if cache.device is not None and cache.device != dev:
        _other_device(cache, dev)
    kp, ks, T, Hkv, D = _rows(k, "k", dev)
    if Hkv != cache.Hkv or D != cache.D:
        raise ValueError(f"k: expected heads ({cache.Hkv}, {cache.D}), got ({Hkv}, {D})")
    Hq = qp = qs = qop = qos = kop = kos = B = vp = vs = tp = te = ts = lp = cp = 0
    csp = max_pos = rot = axes = pp = s0 = s1 = s2 = 0
    if q is not None and q_out is not None:
        qp, qs, n, Hq, qD = _rows(q, "q", dev)
        qop, qos, *like = _rows(q_out, "q_out", dev)
        if like != [n, Hq, qD] or n != T or qD != D:
            raise ValueError(f"q {tuple(q.shape)} and q_out {tuple(q_out.shape)} do not fit k {tuple(k.shape)}")
    elif q is not q_out:
        raise ValueError("q and q_out go together")
    if k_out is not None:
        kop, kos, *like = _rows(k_out, "k_out", dev)
        if like != [T, Hkv, D]:
            raise ValueError(f"k_out {tuple(k_out.shape)} does not fit k {tuple(k.shape)}")
    if cos_sin is not None:
        csp = _flat(cos_sin, "cos_sin", _t_f32, 0, dev)
        max_pos, rot = cos_sin.shape
        shape = pos.shape
        axes = 1 if len(shape) == 1 else shape[0]
        if len(shape) not in (1, 2) or shape[-1] != T or not 1 <= axes <= 3:
            raise ValueError(f"pos: expected ({T},) or (1..3, {T}), got {tuple(pos.shape)}")
        pp = _flat(pos, "pos", i32, axes * T, dev)
        if axes > 1:
            if sections is None or len(sections) != axes:
                raise ValueError(f"sections: expected {axes} numbers of pairs")
            s0, s1, s2 = (*sections, 0)[:3]
    if table is not None:
        vp, vs, *like = _rows(v, "v", dev)
        if like != [T, Hkv, D]:
            raise ValueError(f"v {tuple(v.shape)} does not fit k {tuple(k.shape)}")
        tp, te, ts, B = _table(table, "table", dev)
        lp = _flat(lens, "lens", i32, B, dev)
        if cu is not None:
            cp = _flat(cu, "cu", i32, B + 1, dev)
    a = _pack_rope(symm.world, *cache.packed, T, B, Hq, qp, kp, vp, qs, ks, vs, qop, kop, qos, kos, csp,
                   max_pos, rot, 1 if interleaved else 0, axes, s0, s1, s2, pp, T, cp, tp, te, ts, lp)
    rc = _tdg_rope_append(symm.h, a, _raw_stream(stream, dev))
    if rc:
        _check(rc, "tdg_rope_append")


def prompt_attention(symm: Symm, q, k, v, out, cu_q, cu_k, lse=None, causal=True, scale: float = 0.0,
                     stream=None):
    """Attention over whole prompts packed one after another: q and out (Tq,
    Hq, D), k and v (Tk, Hkv, D), rows possibly strided; cu_q and cu_k (B + 1,)
    int32 row offsets; lse (Tq, Hq) float32 or None."""
    if _torch is None:
        _attn()
    dev, i32 = symm.device, _t_i32
    qp, qs, Tq, Hq, D = _rows(q, "q", dev)
    kp, ks, Tk, Hkv, kD = _rows(k, "k", dev)
    vp, vs, *vlike = _rows(v, "v", dev)
    op, os_, *olike = _rows(out, "out", dev)
    if olike != [Tq, Hq, D] or vlike != [Tk, Hkv, kD] or kD != D:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)} and out "
                         f"{tuple(out.shape)} do not fit together")
    cqp = _flat(cu_q, "cu_q", i32, 1, dev)
    B = cu_q.numel() - 1
    ckp = _flat(cu_k, "cu_k", i32, B + 1, dev)
    lp = 0 if lse is None else _flat(lse, "lse", _t_f32, Tq * Hq, dev)
    a = _pack_prompt(Tq, Tk, B, Hq, Hkv, D, qp, kp, vp, qs, ks, vs, op, os_, lp, cqp, ckp,
                     1 if causal else 0, scale)
    rc = _tdg_prompt_attention(symm.h, a, _raw_stream(stream, dev))
    if rc:
        _check(rc, "tdg_prompt_attention")


def paged_decode_part_bytes(Hq: int, Hkv: int, D: int) -> int:
    return lib().tdg_paged_decode_part_bytes(Hq, Hkv, D)


def paged_decode(symm: Symm, cache: PagedCache, q, out, table, lens, part_off: int, root: int = 0,
                 lse=None, scale: float = 0.0, stream=None):
    """Attention of one new token per sequence over the paged cache: q and out
    (B, Hq, D), rows possibly strided; table (B, entries) int32 page ids; lens
    (B,) int32 lengths with the new token; lse (B, Hq) float32 or None.  The
    partial results (paged_decode_part_bytes) go to region(root) + part_off;
    calls that may overlap, on different streams, need a part_off or root of
    their own."""
    if _torch is None:
        _attn()
    dev = symm.device
    if cache.device is not None and cache.device != dev:
        _other_device(cache, dev)
    qp, qs, B, Hq, D = _rows(q, "q", dev)
    op, os_, *like = _rows(out, "out", dev)
    tp, te, ts, n = _table(table, "table", dev)
    if like != [B, Hq, D] or D != cache.D or n != B:
        raise ValueError(f"q {tuple(q.shape)}, out {tuple(out.shape)} and table {tuple(table.shape)} "
                         f"do not fit together")
    np_ = _flat(lens, "lens", _t_i32, B, dev)
    lp = 0 if lse is None else _flat(lse, "lse", _t_f32, B * Hq, dev)
    a = _pack_decode(symm.world, root, *cache.packed, B, Hq, qp, qs, op, os_, lp, tp, te, ts, np_, part_off, scale)
    rc = _tdg_paged_decode(symm.h, a, _raw_stream(stream, dev))
    if rc:
        _check(rc, "tdg_paged_decode")


def _moe_args(symm, T, H, E, k, x_off, topk_off, gate_off, out_off, recv, counts, base, slot,
              y, row_src, row_tok, row_k, phases):
    import torch
    dev, W = symm.buf.device, symm.world
    rows = W * T * k

    def opt(t, name, dtype, n):
        return None if t is None else _tensor(t, name, dtype, n, dev)
    return MoeArgs(world=W, T=T, H=H, E=E, k=k, x_off=x_off, topk_off=topk_off,
                   gate_off=gate_off, out_off=out_off,
                   recv=opt(recv, "recv", torch.bfloat16, rows * H),
                   y=opt(y, "y", torch.bfloat16, rows * H),
                   counts=opt(counts, "counts", torch.int64, W * E),
                   base=opt(base, "base", torch.int64, E + 1),
                   slot=opt(slot, "slot", torch.int64, rows),
                   row_src=opt(row_src, "row_src", torch.int32, rows),
                   row_tok=opt(row_tok, "row_tok", torch.int32, rows),
                   row_k=opt(row_k, "row_k", torch.int32, rows),
                   workspace=None, workspace_bytes=0, phases=phases)


def moe_workspace_bytes(world: int, T: int, E: int) -> int:
    return lib().tdg_moe_workspace_bytes(world, T, E)


def moe_dispatch_combine(symm: Symm, T: int, H: int, E: int, k: int, x_off: int, topk_off: int,
                         gate_off: int, out_off: int, recv, counts, base, slot, workspace,
                         y=None, row_src=None, row_tok=None, row_k=None, phases=MOE_ALL,
                         stream=None):
    import torch
    _tensor(workspace, "workspace", torch.uint8, 0, symm.buf.device)
    a = _moe_args(symm, T, H, E, k, x_off, topk_off, gate_off, out_off, recv, counts, base, slot,
                  y, row_src, row_tok, row_k, phases)
    a.workspace = workspace.data_ptr()
    a.workspace_bytes = workspace.numel()
    _check(lib().tdg_moe_dispatch_combine(symm.h, ctypes.byref(a), _stream(stream)),
           "tdg_moe_dispatch_combine")


def moe_dispatch_combine_noalloc(symm: Symm, T: int, H: int, E: int, k: int, x_off: int,
                                 topk_off: int, gate_off: int, out_off: int, recv, counts, base,
                                 slot, y=None, row_src=None, row_tok=None, row_k=None,
                                 phases=MOE_ALL, stream=None):
    """Same as moe_dispatch_combine, for callers that cannot allocate device
    memory when they call: the routing scratch is the library's fixed 2 MiB
    device array, so no workspace is passed.  Raises TdgError (TDG_ERR_NOMEM)
    when world * ceil(T/64) * E exceeds 262144."""
    a = _moe_args(symm, T, H, E, k, x_off, topk_off, gate_off, out_off, recv, counts, base, slot,
                  y, row_src, row_tok, row_k, phases)
    _check(lib().tdg_moe_dispatch_combine_noalloc(symm.h, ctypes.byref(a), _stream(stream)),
           "tdg_moe_dispatch_combine_noalloc")


def _blocks(n):
    return -(-n // 128)


def quantise_rows(symm: Symm, x, codes, scale, gated=False, count=None, stream=None):
    """Rows x (n, K) bfloat16 into e4m3 codes (n, K) with a float32 scale for
    each row and block of 128, scale (n, ceil(K / 128)); rows of all three may
    be strided.  gated: x is (n, 2K), gate columns before up columns, and what
    is quantised is silu(gate) * up, to 2^-20 + 2^-23 max(-gate, 0) of it.
    count: int64 tensor whose first element is the number of rows in use
    (base[E:] of the MoE routing); the others are left alone."""
    if _torch is None:
        _attn()
    dev = symm.device
    xp, xs, n, width = _matrix(x, "x", _t_bf16, dev)
    cp, cs, *like = _matrix(codes, "codes", _t_e4m3, dev)
    sp, ss, *slike = _matrix(scale, "scale", _t_f32, dev)
    K = like[1]
    if like[0] != n or width != (2 * K if gated else K) or slike != [n, _blocks(K)]:
        raise ValueError(f"x {tuple(x.shape)}, codes {tuple(codes.shape)} and scale {tuple(scale.shape)} do not fit together")
    np_ = 0 if count is None else _flat(count, "count", _t_i64, 1, dev)
    a = _pack_quantise(QUANT_GATED if gated else QUANT_ROWS, n, K, 1, xp, xs, cp, cs, sp, ss, np_)
    rc = _tdg_quantise(symm.h, a, _raw_stream(stream, dev))
    if rc:
        _check(rc, "tdg_quantise")


def quantise_blocks(symm: Symm, x, codes, scale, stream=None):
    """Weights x (N, K) or (E, N, K) bfloat16 into e4m3 codes of the same shape
    with a float32 scale for each 128 x 128 block, scale (..., ceil(N / 128),
    ceil(K / 128)); all contiguous."""
    if _torch is None:
        _attn()
    dev = symm.device
    xp, cp = _flat(x, "x", _t_bf16, 0, dev), _flat(codes, "codes", _t_e4m3, 0, dev)
    sp = _flat(scale, "scale", _t_f32, 0, dev)
    if x.dim() not in (2, 3):
        raise ValueError(f"x: expected (N, K) or (E, N, K), got {tuple(x.shape)}")
    *E, N, K = x.shape
    if codes.shape != x.shape or tuple(scale.shape) != (*E, _blocks(N), _blocks(K)):
        raise ValueError(f"x {tuple(x.shape)}, codes {tuple(codes.shape)} and scale {tuple(scale.shape)} do not fit together")
    a = _pack_quantise(QUANT_BLOCKS, N, K, E[0] if E else 1, xp, K, cp, K, sp, _blocks(K), 0)
    rc = _tdg_quantise(symm.h, a, _raw_stream(stream, dev))
    if rc:
        _check(rc, "tdg_quantise")


def scaled_gemm(symm: Symm, a, a_scale, b, b_scale, out, base=None, stream=None):
    """out = a @ b.T of 8-bit matrices with a scale for each block of 128 along
    K: a (M, K) e4m3 with a_scale (M, ceil(K / 128)), b (N, K) e4m3 with b_scale
    (ceil(N / 128), ceil(K / 128)), out (M, N) bfloat16 or float32; rows of a,
    a_scale and out may be strided.  base (E + 1,) int64: rows [base[e],
    base[e + 1]) of a go by matrix e of b (E, N, K) and b_scale (E, ...)."""
    if _torch is None:
        _attn()
    dev = symm.device
    ap, as_, M, K = _matrix(a, "a", _t_e4m3, dev)
    sp, ss, *slike = _matrix(a_scale, "a_scale", _t_f32, dev)
    f32 = getattr(out, "dtype", None) is _t_f32
    op, os_, *olike = _matrix(out, "out", _t_f32 if f32 else _t_bf16, dev)
    bp, bsp = _flat(b, "b", _t_e4m3, 0, dev), _flat(b_scale, "b_scale", _t_f32, 0, dev)
    bshape = tuple(b.shape)
    E = 1
    if base is not None:
        E = bshape[0] if len(bshape) == 3 else -1
    N = olike[1]
    lead = () if base is None else (E,)
    if olike[0] != M or slike != [M, _blocks(K)] or bshape != (*lead, N, K) or \
            tuple(b_scale.shape) != (*lead, _blocks(N), _blocks(K)):
        raise ValueError(f"a {tuple(a.shape)}, a_scale {tuple(a_scale.shape)}, b {bshape}, b_scale "
                         f"{tuple(b_scale.shape)} and out {tuple(out.shape)} do not fit together")
    np_ = 0 if base is None else _flat(base, "base", _t_i64, E + 1, dev)
    args = _pack_scaled(M, N, K, E, ap, as_, sp, ss, bp, bsp, op, os_, 1 if f32 else 0, np_)
    rc = _tdg_scaled_gemm(symm.h, args, _raw_stream(stream, dev))
    if rc:
        _check(rc, "tdg_scaled_gemm")


def moe_dispatch_e4m3(symm: Symm, T: int, H: int, k: int, x_off: int, slot, codes, scale, stream=None):
    """The dispatch of moe_dispatch_combine with rows quantised on the way:
    codes (W*T*k, H) e4m3 and scale (W*T*k, ceil(H / 128)) float32 of every
    choice's row, slot (W*T*k) int64 as the routing phase writes it."""
    if _torch is None:
        _attn()
    dev, rows = symm.device, symm.world * T * k
    a = _pack_dispatch_e4m3(symm.world, k, T, H, x_off, _flat(slot, "slot", _t_i64, rows, dev),
                            _flat(codes, "codes", _t_e4m3, rows * H, dev),
                            _flat(scale, "scale", _t_f32, rows * _blocks(H), dev))
    rc = _tdg_moe_dispatch_e4m3(symm.h, a, _raw_stream(stream, dev))
    if rc:
        _check(rc, "tdg_moe_dispatch_e4m3")


def moe_combine_grad(symm: Symm, T: int, H: int, k: int, gate_off: int, dout_off: int, dgate_off: int, slot, y, dy,
                     stream=None):
    """Gradient of the combine: from dout (T, H) bfloat16 at dout_off of every
    region, the gates at gate_off and the experts' outputs y (W*T*k, H), writes
    dy (W*T*k, H) bfloat16 (may be y) and dgate (T, k) float32 at dgate_off."""
    if _torch is None:
        _attn()
    dev, rows = symm.device, symm.world * T * k
    a = _pack_combine_grad(symm.world, k, T, H, gate_off, dout_off, dgate_off, _flat(slot, "slot", _t_i64, rows, dev),
                           _flat(y, "y", _t_bf16, rows * H, dev), _flat(dy, "dy", _t_bf16, rows * H, dev))
    rc = _tdg_moe_combine_grad(symm.h, a, _raw_stream(stream, dev))
    if rc:
        _check(rc, "tdg_moe_combine_grad")


def moe_dispatch_grad(symm: Symm, T: int, H: int, k: int, dx_off: int, slot, drecv, stream=None):
    """Gradient of the dispatch: dx (T, H) bfloat16 at dx_off of every region,
    the sum of the gradients drecv (W*T*k, H) of a token's rows."""
    if _torch is None:
        _attn()
    dev, rows = symm.device, symm.world * T * k
    a = _pack_dispatch_grad(symm.world, k, T, H, dx_off, _flat(slot, "slot", _t_i64, rows, dev),
                            _flat(drecv, "drecv", _t_bf16, rows * H, dev))
    rc = _tdg_moe_dispatch_grad(symm.h, a, _raw_stream(stream, dev))
    if rc:
        _check(rc, "tdg_moe_dispatch_grad")
