"""Lossless BF16 weight codec for B200: Python binding of libdfx (include/dfx.h).

The calls keep the C names and only marshal arguments: pointers are taken from
torch tensors (or passed as integers), streams from ``torch.cuda.Stream``
objects.  Every step of encoding and decoding runs in the CUDA kernels of
``libdfx.so``; there is no CPU fallback, and every call raises
``DfxError`` if the library has not been built (``python -m
lossless_entropy_coded_exponent_b200.build``) or a call fails.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import NamedTuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdfx.so")

DFX_OK = 0
DFX_ERR_ARG = 1
DFX_ERR_CAPACITY = 2
DFX_ERR_CORRUPT = 3
DFX_ERR_TOO_LARGE = 4
DFX_ERR_CUDA = 5
DFX_ERR_UNSUPPORTED = 6

DFX_STATUS_HEADER = 0x1
DFX_STATUS_TABLE = 0x2
DFX_STATUS_INDEX = 0x4
DFX_STATUS_STREAM = 0x8
DFX_STATUS_TIMEOUT = 0x10
DFX_INJECT_SKIP_SLICE_COPY = 0x1
DFX_INJECT_SKIP_TILE_COPY = 0x4
DFX_CODER_HUFFMAN = 0
DFX_CODER_TANS = 1
DFX_CODER_TANS2 = 2  # tANS with two interleaved states per chunk
DFX_DECODE_EARLY_READ = 0x1
DFX_F32 = 0
DFX_BF16 = 1
DFX_SCORE_SOFTMAX = 0
DFX_SCORE_SIGMOID = 1
DFX_QUANT_SWIGLU = 0x1

# The exported C symbols, in include/dfx.h order.
EXPORTS = (
    "dfx_version",
    "dfx_strerror",
    "dfx_container_layout",
    "dfx_plan",
    "dfx_encode",
    "dfx_decode",
    "dfx_decode_range",
    "dfx_decode_host",
    "dfx_decode_gemm",
    "dfx_decode_batch",
    "dfx_device_status",
    "dfx_free",
    "dfx_encode_static",
    "dfx_debug_inject",
    "dfx_route_workspace",
    "dfx_route",
    "dfx_quantize_fp8",
    "dfx_gemm_fp8",
    "dfx_combine",
)


class DfxError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {dfx_strerror(code) if _lib_handle else code} (code {code})")
        self.code = code


class dfx_params(ctypes.Structure):
    _fields_ = [("chunk_symbols", ctypes.c_uint32), ("group_chunks", ctypes.c_uint32), ("max_len", ctypes.c_uint32),
                ("coder", ctypes.c_uint32), ("table_log", ctypes.c_uint32), ("decode_flags", ctypes.c_uint32)]


class dfx_layout(ctypes.Structure):
    _fields_ = [(name, ctypes.c_uint64) for name in
                ("n", "n_chunk", "n_group", "off_len", "off_gbase", "off_clen", "off_m", "off_stream",
                 "stream_bytes", "total_bytes")]


class dfx_route_params(ctypes.Structure):
    _fields_ = [("score", ctypes.c_uint32), ("topk", ctypes.c_uint32), ("groups", ctypes.c_uint32),
                ("top_groups", ctypes.c_uint32), ("group_best", ctypes.c_uint32), ("renormalize", ctypes.c_uint32),
                ("scale", ctypes.c_float)]


_lib_handle = None


def lib() -> ctypes.CDLL:
    """The loaded libdfx.so; raises if it has not been built."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libdfx.so is missing at {LIB_PATH}: build it with "
                "`python -m lossless_entropy_coded_exponent_b200.build` (there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        vp = ctypes.c_void_p
        L.dfx_version.argtypes = []
        L.dfx_version.restype = ctypes.c_uint32
        L.dfx_strerror.argtypes = [ctypes.c_int]
        L.dfx_strerror.restype = ctypes.c_char_p
        L.dfx_container_layout.argtypes = [ctypes.c_uint64, ctypes.POINTER(dfx_params), ctypes.c_uint64,
                                           ctypes.POINTER(dfx_layout)]
        L.dfx_plan.argtypes = [ctypes.POINTER(vp), ctypes.c_uint64, ctypes.POINTER(dfx_params),
                               ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]
        L.dfx_encode.argtypes = [vp, vp, vp, ctypes.c_size_t, vp, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t), vp]
        L.dfx_decode.argtypes = [vp, vp, ctypes.c_size_t, vp, vp]
        L.dfx_decode_range.argtypes = [vp, vp, ctypes.c_size_t, ctypes.c_uint64, ctypes.c_uint64, vp, vp]
        L.dfx_decode_host.argtypes = [vp, vp, ctypes.c_size_t, vp, ctypes.c_size_t, vp, ctypes.c_uint32, vp, vp]
        L.dfx_decode_gemm.argtypes = [vp, vp, ctypes.c_size_t, ctypes.c_uint64, ctypes.c_uint64, vp, ctypes.c_uint32, vp,
                                      vp, vp]
        L.dfx_decode_batch.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(ctypes.c_size_t),
                                       ctypes.POINTER(vp), ctypes.c_uint32, vp]
        L.dfx_device_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
        L.dfx_free.argtypes = [vp]
        L.dfx_debug_inject.argtypes = [ctypes.c_uint32]
        L.dfx_encode_static.argtypes = [vp, ctypes.c_uint64, ctypes.POINTER(dfx_params), vp, ctypes.c_size_t,
                                        ctypes.POINTER(ctypes.c_size_t), vp]
        u64, u32, sz = ctypes.c_uint64, ctypes.c_uint32, ctypes.c_size_t
        rp = ctypes.POINTER(dfx_route_params)
        L.dfx_route_workspace.argtypes = [u64, u32, rp, ctypes.POINTER(sz)]
        L.dfx_route.argtypes = [vp, vp, u32, u64, u64, u32, vp, rp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.dfx_quantize_fp8.argtypes = [vp, vp, u32, u64, u64, vp, u64, u64, u32, u32, vp, u64, vp, u64, vp]
        L.dfx_gemm_fp8.argtypes = [vp, vp, u64, vp, u64, u64, vp, u64, vp, u64, u64, u64, u32, vp, vp, u32, u64, vp]
        L.dfx_combine.argtypes = [vp, vp, u32, u64, u64, u64, vp, vp, u64, u32, vp, u32, u64, vp]
        for f in ("dfx_container_layout", "dfx_plan", "dfx_encode", "dfx_decode", "dfx_decode_range", "dfx_decode_host",
                  "dfx_decode_gemm", "dfx_decode_batch",
                  "dfx_device_status", "dfx_free", "dfx_encode_static", "dfx_debug_inject", "dfx_route_workspace",
                  "dfx_route", "dfx_quantize_fp8", "dfx_gemm_fp8", "dfx_combine"):
            getattr(L, f).restype = ctypes.c_int
        _lib_handle = L
    return _lib_handle


def _check(rc: int, what: str) -> None:
    if rc != DFX_OK:
        raise DfxError(rc, what)


def _ptr(x) -> int | None:
    """Device pointer of a tensor, or an integer address as is."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s) -> int | None:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _params(chunk_symbols=0, group_chunks=0, max_len=0, coder=DFX_CODER_HUFFMAN, table_log=0, decode_flags=0):
    return dfx_params(chunk_symbols, group_chunks, max_len, coder, table_log, decode_flags)


def dfx_version() -> int:
    return int(lib().dfx_version())


def dfx_strerror(code: int) -> str:
    return lib().dfx_strerror(code).decode()


def dfx_container_layout(n: int, total_bits: int, chunk_symbols=0, group_chunks=0, max_len=0,
                         coder=DFX_CODER_HUFFMAN, table_log=0) -> dict:
    out = dfx_layout()
    p = _params(chunk_symbols, group_chunks, max_len, coder, table_log)
    _check(lib().dfx_container_layout(n, ctypes.byref(p), total_bits, ctypes.byref(out)), "dfx_container_layout")
    return {name: int(getattr(out, name)) for name, _ in dfx_layout._fields_}


class Plan:
    """An open dfx plan (the C ``dfx_plan_t``) plus the sizes dfx_plan reported."""

    def __init__(self, handle: int, n: int, max_compressed_bytes: int, workspace_bytes: int, params: tuple):
        self.handle = handle
        self.n = n
        self.max_compressed_bytes = max_compressed_bytes
        self.workspace_bytes = workspace_bytes
        self.params = params

    def free(self) -> None:
        if self.handle:
            _check(lib().dfx_free(self.handle), "dfx_free")
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.free()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def dfx_plan(n: int, chunk_symbols: int = 0, group_chunks: int = 0, max_len: int = 0,
             coder: int = DFX_CODER_HUFFMAN, table_log: int = 0, decode_flags: int = 0) -> Plan:
    h = ctypes.c_void_p()
    mx = ctypes.c_size_t()
    ws = ctypes.c_size_t()
    p = _params(chunk_symbols, group_chunks, max_len, coder, table_log, decode_flags)
    _check(lib().dfx_plan(ctypes.byref(h), n, ctypes.byref(p), ctypes.byref(mx), ctypes.byref(ws)), "dfx_plan")
    return Plan(h.value, n, mx.value, ws.value, (chunk_symbols, group_chunks, max_len, coder, table_log))


def dfx_encode(plan: Plan, d_bf16, d_out, out_capacity: int, d_workspace, workspace_bytes: int,
               want_size: bool = False, stream=None) -> int | None:
    size = ctypes.c_size_t()
    rc = lib().dfx_encode(plan.handle, _ptr(d_bf16), _ptr(d_out), out_capacity, _ptr(d_workspace), workspace_bytes,
                          ctypes.byref(size) if want_size else None, _stream(stream))
    _check(rc, "dfx_encode")
    return size.value if want_size else None


def dfx_decode(plan: Plan, d_comp, comp_bytes: int, d_bf16, stream=None) -> None:
    _check(lib().dfx_decode(plan.handle, _ptr(d_comp), comp_bytes, _ptr(d_bf16), _stream(stream)), "dfx_decode")


DEFAULT_CHUNK_SYMBOLS = 128  # dfx_params.chunk_symbols = 0 means this (include/dfx.h)


def group_elements(plan: Plan) -> int:
    """Elements per group of the plan's containers (32 chunks of chunk_symbols)."""
    return 32 * (plan.params[0] or DEFAULT_CHUNK_SYMBOLS)


def dfx_decode_range(plan: Plan, d_comp, comp_bytes: int, first_group: int, group_count: int, d_bf16,
                     stream=None) -> None:
    """Decode groups [first_group, first_group + group_count) into d_bf16 (which holds
    element first_group * 32 * chunk_symbols at index 0)."""
    _check(lib().dfx_decode_range(plan.handle, _ptr(d_comp), comp_bytes, first_group, group_count, _ptr(d_bf16),
                                  _stream(stream)), "dfx_decode_range")


def dfx_decode_host(plan: Plan, h_comp, comp_bytes: int, d_staging, staging_bytes: int, d_bf16, slices: int = 0,
                    copy_stream=None, decode_stream=None) -> None:
    """Stream a container in (pinned) host memory to d_staging slice by slice while
    decoding the slices into d_bf16 (copies on copy_stream, decoding on decode_stream)."""
    _check(lib().dfx_decode_host(plan.handle, _ptr(h_comp), comp_bytes, _ptr(d_staging), staging_bytes,
                                 _ptr(d_bf16), slices, _stream(copy_stream), _stream(decode_stream)),
           "dfx_decode_host")


def dfx_decode_gemm(plan: Plan, d_comp, comp_bytes: int, rows: int, cols: int, d_x, tokens: int, d_y,
                    d_w_out=None, stream=None) -> None:
    """Y = X W^T with W (rows x cols BF16) decoded from its container inside the GEMM
    kernel; X tokens x cols BF16, Y tokens x rows FP32; d_w_out (optional) also
    receives the decoded W."""
    _check(lib().dfx_decode_gemm(plan.handle, _ptr(d_comp), comp_bytes, rows, cols, _ptr(d_x), tokens, _ptr(d_y),
                                 _ptr(d_w_out), _stream(stream)), "dfx_decode_gemm")


def dfx_decode_batch(plans, d_comps, comp_bytes, d_bf16s, stream=None) -> None:
    """Decode several containers with one kernel launch (sequences of equal length)."""
    n = len(plans)
    if not (len(d_comps) == len(comp_bytes) == len(d_bf16s) == n):
        raise ValueError("dfx_decode_batch: plans, containers, sizes and outputs differ in length")
    vp = ctypes.c_void_p
    hp = (vp * max(n, 1))(*[p.handle if p is not None else None for p in plans])
    cp = (vp * max(n, 1))(*[_ptr(c) for c in d_comps])
    sz = (ctypes.c_size_t * max(n, 1))(*[int(b) for b in comp_bytes])
    op = (vp * max(n, 1))(*[_ptr(o) for o in d_bf16s])
    _check(lib().dfx_decode_batch(hp, cp, sz, op, n, _stream(stream)), "dfx_decode_batch")


def dfx_debug_inject(flags: int) -> None:
    """Test hook: DFX_INJECT_SKIP_SLICE_COPY makes later decodes leave one stream-slice
    copy out so that a bounded wait runs out (status DFX_STATUS_TIMEOUT); 0 restores."""
    _check(lib().dfx_debug_inject(flags), "dfx_debug_inject")


def dfx_device_status(plan: Plan, stream=None) -> int:
    v = ctypes.c_uint32()
    _check(lib().dfx_device_status(plan.handle, _stream(stream), ctypes.byref(v)), "dfx_device_status")
    return int(v.value)


def dfx_free(plan: Plan) -> None:
    plan.free()


def dfx_encode_static(d_bf16, n: int, d_out, out_capacity: int, want_size: bool = False, stream=None,
                      chunk_symbols: int = 0, group_chunks: int = 0, max_len: int = 0,
                      coder: int = DFX_CODER_HUFFMAN) -> int | None:
    """Encode without any device allocation by the library (no plan, no workspace);
    for callers whose device memory is owned by another allocator (coder 0 only)."""
    size = ctypes.c_size_t()
    p = _params(chunk_symbols, group_chunks, max_len, coder)
    rc = lib().dfx_encode_static(_ptr(d_bf16), n, ctypes.byref(p), _ptr(d_out), out_capacity,
                                 ctypes.byref(size) if want_size else None, _stream(stream))
    _check(rc, "dfx_encode_static")
    return size.value if want_size else None


def dfx_route_workspace(tokens: int, experts: int, params: dfx_route_params) -> int:
    size = ctypes.c_size_t()
    _check(lib().dfx_route_workspace(tokens, experts, ctypes.byref(params), ctypes.byref(size)), "dfx_route_workspace")
    return size.value


def dfx_route(plan: Plan, d_logits, logits_type: int, ld_logits: int, tokens: int, experts: int, d_bias,
              params: dfx_route_params, d_ids, d_weights, d_offsets=None, d_rows=None, d_slots=None, d_workspace=None,
              workspace_bytes: int = 0, stream=None) -> None:
    """Each token's best experts and their weights; with d_offsets, d_rows and d_slots also
    the assignments sorted by expert."""
    _check(lib().dfx_route(plan.handle, _ptr(d_logits), logits_type, ld_logits, tokens, experts, _ptr(d_bias),
                           ctypes.byref(params), _ptr(d_ids), _ptr(d_weights), _ptr(d_offsets), _ptr(d_rows),
                           _ptr(d_slots), _ptr(d_workspace), workspace_bytes, _stream(stream)), "dfx_route")


def dfx_quantize_fp8(plan: Plan, d_x, x_type: int, ld_x: int, x_rows: int, d_index, rows: int, cols: int,
                     block_rows: int, flags: int, d_q, ld_q: int, d_scales, ld_scales: int, stream=None) -> None:
    """e4m3 values and e8m0 scales of 1x128 (block_rows 1) or 128x128 (128) blocks."""
    _check(lib().dfx_quantize_fp8(plan.handle, _ptr(d_x), x_type, ld_x, x_rows, _ptr(d_index), rows, cols, block_rows,
                                  flags, _ptr(d_q), ld_q, _ptr(d_scales), ld_scales, _stream(stream)),
           "dfx_quantize_fp8")


def dfx_gemm_fp8(plan: Plan, d_x, ld_x: int, d_x_scales, ld_x_scales: int, tokens: int, d_w, ld_w: int, d_w_scales,
                 ld_w_scales: int, rows: int, cols: int, experts: int, d_offsets, d_y, y_type: int, ld_y: int,
                 stream=None) -> None:
    """Y = X W^T of dfx_quantize_fp8's operands, with one matrix or one per expert (d_offsets)."""
    _check(lib().dfx_gemm_fp8(plan.handle, _ptr(d_x), ld_x, _ptr(d_x_scales), ld_x_scales, tokens, _ptr(d_w), ld_w,
                              _ptr(d_w_scales), ld_w_scales, rows, cols, experts, _ptr(d_offsets), _ptr(d_y), y_type,
                              ld_y, _stream(stream)), "dfx_gemm_fp8")


def dfx_combine(plan: Plan, d_z, z_type: int, ld_z: int, z_rows: int, cols: int, d_slots, d_weights, tokens: int,
                topk: int, d_y, y_type: int, ld_y: int, stream=None) -> None:
    """y[t] = sum over k of weights[t, k] z[slots[t, k]]."""
    _check(lib().dfx_combine(plan.handle, _ptr(d_z), z_type, ld_z, z_rows, cols, _ptr(d_slots), _ptr(d_weights), tokens,
                             topk, _ptr(d_y), y_type, ld_y, _stream(stream)), "dfx_combine")


# ---------------------------------------------------------------- tensor helpers
# Allocation goes through torch; the work is the C calls above.

def encode(x, plan: Plan | None = None, stream=None, **params):
    """Compress a CUDA tensor of BF16 (or int16/uint16 bit patterns); returns the
    container as a uint8 CUDA tensor trimmed to its size (synchronises `stream`)."""
    import torch

    flat = x.reshape(-1)
    own = plan is None
    plan = plan or dfx_plan(flat.numel(), **params)
    try:
        out = torch.empty(plan.max_compressed_bytes, dtype=torch.uint8, device=flat.device)
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=flat.device)
        size = dfx_encode(plan, flat, out, out.numel(), ws, ws.numel(), want_size=True, stream=stream)
        return out[:size].clone()
    finally:
        if own:
            plan.free()


def decode(comp, n: int, plan: Plan | None = None, out=None, stream=None, check: bool = True, **params):
    """Decode a container (uint8 CUDA tensor) into a BF16 CUDA tensor of n elements.
    With check=True the stream is synchronised and a corrupt container raises."""
    import torch

    own = plan is None
    plan = plan or dfx_plan(n, **params)
    try:
        if out is None:
            out = torch.empty(n, dtype=torch.bfloat16, device=comp.device)
        dfx_decode(plan, comp, comp.numel(), out, stream=stream)
        if check:
            st = dfx_device_status(plan, stream=stream)
            if st:
                raise DfxError(DFX_ERR_CORRUPT, f"dfx_decode (device status 0x{st:x})")
        return out
    finally:
        if own:
            plan.free()


# Layers of experts with 8-bit weights.  These run on the tensors' device and on its current
# torch stream (or `stream`, a torch stream: then what they allocate belongs to it, and the memory of
# their tensors is not given to others before its work on them is done; the caller lets it wait for
# the work that makes them).  A plan of the device may be passed in; without one a call makes its own, waits for the work and raises
# if its status word says that an index was out of range or a wait ran out.

class Fp8(NamedTuple):
    """e4m3 values and e8m0 block scales (include/dfx.h): uint8 tensors [..., rows, ld]."""
    values: "torch.Tensor"
    scales: "torch.Tensor"
    cols: int         # values of a row
    block_rows: int   # 1, or 128 (weights)


class Routing(NamedTuple):
    """What dfx_route gives: experts and weights [tokens, topk]; where the assignments of each
    expert begin [experts + 1], their tokens [tokens * topk], and each assignment's place."""
    ids: "torch.Tensor"
    weights: "torch.Tensor"
    offsets: "torch.Tensor"
    rows: "torch.Tensor"
    slots: "torch.Tensor"


@contextlib.contextmanager
def _call(tensors, plan, stream, what):
    """Device, stream and plan of a helper's calls on `tensors` (or None among them): yields
    (plan, stream handle)."""
    import torch

    tensor = tensors[0]
    if not tensor.is_cuda:
        raise ValueError(f"{what}: tensors must be on a CUDA device (there is no CPU fallback)")
    if stream is not None and stream.device != tensor.device:
        raise ValueError(f"{what}: a stream of {stream.device} for tensors on {tensor.device}")
    with torch.cuda.device(tensor.device), torch.cuda.stream(stream):
        if stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        handle = torch.cuda.current_stream().cuda_stream
        own = plan is None
        if own:
            plan = dfx_plan(0)
        try:
            yield plan, handle
            if own:
                st = dfx_device_status(plan, stream=handle)
                if st:
                    raise DfxError(DFX_ERR_CORRUPT, f"{what} (device status 0x{st:x})")
        finally:
            if own:
                plan.free()


def _float_type(t, what: str) -> int:
    import torch

    if t not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{what}: float32 or bfloat16, not {t}")
    return DFX_F32 if t == torch.float32 else DFX_BF16


def _matrix(x, what: str):
    """A 2-D tensor whose rows the library can read: neighbouring elements, 16-byte aligned."""
    if x.dim() != 2:
        raise ValueError(f"{what}: a matrix is needed, not {x.dim()} dimensions")
    return x if x.stride(1) == 1 and x.stride(0) >= x.shape[1] and x.data_ptr() % 16 == 0 else x.clone(
        memory_format=_contiguous())


def _contiguous():
    import torch

    return torch.contiguous_format


def _ld(x) -> int:
    return max(x.stride(0), x.shape[1])


def _whole_fp8(f: Fp8, what: str):
    """Refuses an Fp8 whose tensors are not laid out as its rows and columns say."""
    import torch

    rows, blocks = f.values.shape[-2], -(-f.cols // 128)
    if f.values.dtype != torch.uint8 or f.scales.dtype != torch.uint8:
        raise TypeError(f"{what}: values and scales are uint8 tensors")
    if not f.values.is_contiguous() or not f.scales.is_contiguous() or f.values.shape[:-2] != f.scales.shape[:-2] \
            or f.scales.shape[-2] != -(-rows // f.block_rows) or f.values.shape[-1] < f.cols or f.scales.shape[-1] < blocks:
        raise ValueError(f"{what}: values and scales are contiguous, with a row of scales for {f.block_rows} of values")


def _same_device(what: str, *tensors):
    if len({t.device for t in tensors if t is not None}) > 1:
        raise ValueError(f"{what}: tensors on different devices")


def route(logits, topk: int, score: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
          group_best: int = 1, renormalize: bool = False, scale: float = 1.0, plan: Plan | None = None,
          stream=None) -> Routing:
    """Each token's best experts (dfx_route) from gate logits [tokens, experts].  scale: a factor of
    every weight (0 counts as 1)."""
    import torch

    if score not in ("softmax", "sigmoid"):
        raise ValueError("route: score is 'softmax' or 'sigmoid'")
    kind = _float_type(logits.dtype, "route")
    _same_device("route", logits, bias)
    with _call((logits, bias), plan, stream, "route") as (p, s):
        x = _matrix(logits, "route")
        tokens, experts = x.shape
        if bias is not None:
            if bias.shape != (experts,):
                raise ValueError("route: a bias for each expert")
            bias = bias.to(torch.float32).clone()  # aligned, whatever it was a part of
        params = dfx_route_params(score=DFX_SCORE_SIGMOID if score == "sigmoid" else DFX_SCORE_SOFTMAX, topk=topk,
                                  groups=groups, top_groups=top_groups, group_best=group_best,
                                  renormalize=int(renormalize), scale=scale)
        ints = lambda *shape: torch.empty(shape, dtype=torch.int32, device=x.device)  # noqa: E731
        work = torch.empty(dfx_route_workspace(tokens, experts, params), dtype=torch.uint8, device=x.device)
        out = Routing(ints(tokens, topk), torch.empty(tokens, topk, device=x.device), ints(experts + 1),
                      ints(tokens * topk), ints(tokens, topk))
        dfx_route(p, x, kind, _ld(x), tokens, experts, bias, params, *out, work, work.numel(), stream=s)
    return out


def quantize_fp8(x, block_rows: int = 1, index=None, swiglu: bool = False, plan: Plan | None = None,
                 stream=None) -> Fp8:
    """e4m3 values and block scales (dfx_quantize_fp8) of x [rows, cols], or of each matrix of
    x [experts, rows, cols].  index (int32): output row r is x[index[r]], a row with a negative
    index is not written; swiglu: x holds gates, then values, in each row."""
    import torch

    kind = _float_type(x.dtype, "quantize_fp8")
    if x.dim() not in (2, 3) or (x.dim() == 3 and (index is not None or swiglu)):
        raise ValueError("quantize_fp8: a matrix, or several of them without index and swiglu")
    if swiglu and x.shape[-1] % 2:
        raise ValueError("quantize_fp8: as many gates as values")
    if index is not None and (index.dim() != 1 or index.dtype != torch.int32):
        raise TypeError("quantize_fp8: index is a vector of int32")
    _same_device("quantize_fp8", x, index)
    cols = x.shape[-1] // 2 if swiglu else x.shape[-1]
    rows = x.shape[-2] if index is None else index.numel()
    blocks = -(-cols // 128)
    with _call((x, index), plan, stream, "quantize_fp8") as (p, s):
        q = torch.empty(*x.shape[:-2], rows, -(-cols // 16) * 16, dtype=torch.uint8, device=x.device)
        # rows of scales in 16-byte pieces, which the product loads faster
        sc = torch.empty(*x.shape[:-2], -(-rows // block_rows), -(-blocks // 16) * 16, dtype=torch.uint8, device=x.device)
        if index is not None:
            index = index if index.is_contiguous() and index.data_ptr() % 16 == 0 else index.clone()
        for part, pq, ps in zip(x, q, sc) if x.dim() == 3 else ((x, q, sc),):
            m = _matrix(part, "quantize_fp8")
            dfx_quantize_fp8(p, m, kind, _ld(m), m.shape[0], index, rows, cols, block_rows,
                             DFX_QUANT_SWIGLU if swiglu else 0, pq, q.shape[-1], ps, sc.shape[-1], stream=s)
    return Fp8(q, sc, cols, block_rows)


def gemm_fp8(x: Fp8, w: Fp8, offsets=None, dtype=None, out=None, plan: Plan | None = None, stream=None):
    """x w^T (dfx_gemm_fp8): x [tokens, cols]; w [rows, cols], or [experts, rows, cols] with
    offsets (int32 [experts + 1]): expert e has x's rows offsets[e] .. offsets[e + 1] - 1, and rows
    that no expert has are not written.  dtype: bfloat16 (default) or float32; out: a matrix to
    write into."""
    import torch

    if x.block_rows != 1 or w.block_rows != 128 or x.values.dim() != 2 or w.values.dim() not in (2, 3):
        raise ValueError("gemm_fp8: x in blocks of 1 x 128, w in blocks of 128 x 128")
    if x.cols != w.cols:
        raise ValueError(f"gemm_fp8: rows of {x.cols} and of {w.cols} values")
    _whole_fp8(x, "gemm_fp8")
    _whole_fp8(w, "gemm_fp8")
    experts = w.values.shape[0] if w.values.dim() == 3 else 1
    if offsets is not None and (offsets.dtype != torch.int32 or offsets.shape != (experts + 1,) or not offsets.is_contiguous()):
        raise ValueError("gemm_fp8: offsets is an int32 vector of one more than the experts")
    _same_device("gemm_fp8", x.values, x.scales, w.values, w.scales, offsets, out)
    if out is not None and (out.dim() != 2 or out.stride(1) != 1 or (out.shape[0] > 1 and out.stride(0) < out.shape[1])
                            or out.shape != (x.values.shape[0], w.values.shape[-2])
                            or (dtype is not None and out.dtype != dtype)):
        raise ValueError("gemm_fp8: out is a [tokens, rows] matrix with neighbouring elements")
    dtype = out.dtype if out is not None else dtype or torch.bfloat16
    kind = _float_type(dtype, "gemm_fp8")
    with _call((*x[:2], *w[:2], offsets, out), plan, stream, "gemm_fp8") as (p, s):
        tokens, rows = x.values.shape[0], w.values.shape[-2]
        y = torch.empty(tokens, rows, dtype=dtype, device=x.values.device) if out is None else out
        dfx_gemm_fp8(p, x.values, x.values.shape[-1], x.scales, x.scales.shape[-1], tokens, w.values, w.values.shape[-1],
                     w.scales, w.scales.shape[-1], rows, x.cols, experts, offsets, y, kind, _ld(y), stream=s)
    return y


def combine(z, slots, weights, dtype=None, plan: Plan | None = None, stream=None):
    """y[t] = sum over k of weights[t, k] z[slots[t, k]] (dfx_combine); a negative slot adds
    nothing.  dtype: that of z (default), bfloat16 or float32."""
    import torch

    dtype = dtype or z.dtype
    kind, y_kind = _float_type(z.dtype, "combine"), _float_type(dtype, "combine")
    if slots.shape != weights.shape or slots.dim() != 2 or slots.dtype != torch.int32 or weights.dtype != torch.float32:
        raise ValueError("combine: int32 slots and float32 weights [tokens, topk]")
    _same_device("combine", z, slots, weights)
    with _call((z, slots, weights), plan, stream, "combine") as (p, s):
        m = _matrix(z, "combine")
        slots, weights = (t if t.is_contiguous() and t.data_ptr() % 16 == 0 else t.clone(memory_format=_contiguous())
                          for t in (slots, weights))
        y = torch.empty(slots.shape[0], m.shape[1], dtype=dtype, device=z.device)
        dfx_combine(p, m, kind, _ld(m), m.shape[0], m.shape[1], slots, weights, slots.shape[0], slots.shape[1], y, y_kind,
                    _ld(y), stream=s)
    return y


def experts_fp8(x, logits, w_in: Fp8, w_out: Fp8, topk: int, plan: Plan | None = None, stream=None, **routing):
    """A mixture-of-experts feed-forward layer with 8-bit weights: for each token the weighted sum
    over its experts of w_out (silu(gate) * value), where [gate, value] = w_in x.
      x [tokens, width], logits [tokens, experts] (a row of -inf: padding, zeros come out);
      w_in: quantize_fp8 of [experts, 2 * inner, width] in 128-row blocks (gates first), w_out of
      [experts, width, inner]; routing: route's keywords.  The result has x's type."""
    import torch

    if x.dim() != 2 or logits.dim() != 2 or x.shape[0] != logits.shape[0]:
        raise ValueError("experts_fp8: x [tokens, width] and logits [tokens, experts] of the same tokens")
    for w, shape in ((w_in, (2 * w_out.cols, x.shape[1])), (w_out, (x.shape[1], w_out.cols))):
        _whole_fp8(w, "experts_fp8")
        if w.block_rows != 128 or w.values.dim() not in (2, 3) or (w.values.shape[-2], w.cols) != shape \
                or w.values.shape[:-2].numel() != logits.shape[1]:
            raise ValueError("experts_fp8: w_in [experts, 2 * inner, width] and w_out [experts, width, inner] in blocks of "
                             "128 rows, a matrix for each column of logits")
    tensors = (x, logits, *w_in[:2], *w_out[:2], routing.get("bias"))
    _same_device("experts_fp8", *tensors)
    with _call(tensors, plan, stream, "experts_fp8") as (p, _):
        r = route(logits, topk, plan=p, **routing)
        # the tokens in the experts' order, an expert's rows beside one another
        xq = quantize_fp8(x, index=r.rows, plan=p)
        h = gemm_fp8(xq, w_in, r.offsets, dtype=torch.bfloat16, plan=p)
        hq = quantize_fp8(h, swiglu=True, plan=p)
        z = gemm_fp8(hq, w_out, r.offsets, dtype=torch.bfloat16, plan=p)
        return combine(z, r.slots, r.weights, dtype=x.dtype, plan=p)
