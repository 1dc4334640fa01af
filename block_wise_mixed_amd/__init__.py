"""Block-wise mixed-precision weight-only quantized matmul for MI355X (gfx950).

Thin ctypes binding over the C ABI of libmsq.so (include/msq.h).  This module
only marshals arguments: every step of quantize-pack and of y = x . W^T runs
in the library's HIP kernels.  PyTorch provides device memory and the current
stream.  There is no fallback: if libmsq.so is missing every call raises.

    pw = quantize_pack(W_bf16_cuda, bits, perm_row, perm_col)   # offline
    y  = gemm(x_bf16_cuda, pw)                                   # fp32 [M][N]

Method: a bf16 weight is reordered in rows and columns, cut into 64x128
blocks with a bitwidth from {0,1,2,3,4,8} each, and every block row-group of
128 is round-to-nearest quantized with its own scale and zero point
("ScaleBITS" summary page, sections Approach and Limitations).
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from dataclasses import dataclass
from typing import Optional

import numpy as np

__all__ = ["MsqError", "PackedWeight", "plan", "quantize_pack", "allocate_packed", "pack_into",
           "pack_bytes", "gemm", "workspace_bytes",
           "OPTION_FIELDS", "gemm_noalloc", "NOALLOC_SCRATCH_BYTES",
           "gemm_group", "group_workspace_bytes", "GROUP_MAX",
           "library_path", "load_library", "KERNELS", "FORMAT_VERSION", "GEMV_MAX_M",
           "allocate_bits", "alloc_workspace_bytes", "ALLOC_LEVELS", "reorder_channels",
           "KVCache", "allocate_kv_cache", "kv_write", "kv_read", "kv_attention",
           "kv_attention_workspace_bytes", "kv_attention_plan", "KV_HEAD_DIMS", "KV_BLOCK_TOKENS"]

FORMAT_VERSION = 2
GEMV_MAX_M = 64
KERNELS = {"auto": 0, "gemv": 1, "gemm": 2}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libmsq.so"
_lib = None


def library_path() -> str:
    return os.environ.get("MSQ_LIBRARY", os.path.join(_HERE, _LIB_NAME))


class MsqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        text = _lib.msq_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{where}: msq status {status} ({text})")


class _Sizes(ctypes.Structure):
    _fields_ = [("code_bytes", ctypes.c_int64), ("scale_bytes", ctypes.c_int64),
                ("zero_bytes", ctypes.c_int64), ("offset_bytes", ctypes.c_int64),
                ("blocks_per_bits", ctypes.c_int64 * 17), ("mean_bits", ctypes.c_double)]


class _Options(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("gemv_split", ctypes.c_int32),
                ("gemv_waves", ctypes.c_int32), ("m1_prep", ctypes.c_int32),
                ("gemm_split", ctypes.c_int32)]


OPTION_FIELDS = ("gemv_split", "gemv_waves", "m1_prep", "gemm_split")


def _options(kernel: str = "auto", options: Optional[dict] = None) -> Optional[_Options]:
    """msq_options for a kernel name and a dict of launch choices (None: automatic)."""
    if kernel == "auto" and not options:
        return None
    o = _Options()
    o.kernel = KERNELS[kernel]
    for k, v in (options or {}).items():
        if k not in OPTION_FIELDS:
            raise ValueError(f"unknown option {k!r}; known: {OPTION_FIELDS}")
        setattr(o, k, int(v))
    return o


class _Weight(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("bits", ctypes.c_void_p), ("perm_row", ctypes.c_void_p),
                ("perm_col", ctypes.c_void_p), ("block_offset", ctypes.c_void_p),
                ("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("zero", ctypes.c_void_p), ("code_bytes", ctypes.c_int64),
                ("tile16_blocks", ctypes.c_int64)]


class _KvCache(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_tokens", ctypes.c_int32),
                ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class _KvSeqs(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("table_width", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("offset", ctypes.c_void_p),
                ("total", ctypes.c_int64), ("max_count", ctypes.c_int32)]


class _KvAttn(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_token_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64), ("q_dtype", ctypes.c_int32),
                ("q_heads", ctypes.c_int32), ("kv_len", ctypes.c_void_p),
                ("max_kv_len", ctypes.c_int64), ("scale", ctypes.c_float),
                ("causal", ctypes.c_int32), ("window", ctypes.c_int32),
                ("out", ctypes.c_void_p), ("out_dtype", ctypes.c_int32),
                ("lse", ctypes.c_void_p)]


class _KvPlan(ctypes.Structure):
    _fields_ = [("tile_rows", ctypes.c_int32), ("wavefronts", ctypes.c_int32),
                ("parts", ctypes.c_int32), ("join", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_size_t)]


_KV_CACHE = struct.Struct("@qiiiPPPP")  # the fields of _KvCache
_KV_SEQS = struct.Struct("@iiPPqi")  # the fields of _KvSeqs
_KV_ATTN = struct.Struct("@PqqiiPqfiiPiP")  # the fields of _KvAttn
_KV_CACHE_FIELDS = frozenset(("num_blocks", "kv_heads", "head_dim", "block_tokens", "k_codes",
                              "v_codes", "k_scale", "v_scale"))


def _pack(fields: struct.Struct, to, what: str, *values) -> None:
    """All fields of a ctypes structure at once (a third of the time that its constructor takes);
    values that do not fit raise instead of wrapping around.  (The calls do the same in place.)"""
    try:
        fields.pack_into(to, 0, *values)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"{what}: {e}") from None


def load_library():
    """Load libmsq.so once; raises OSError with the path if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise OSError(f"{path} not found: build it with `python -m block_wise_mixed_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    lib.msq_plan.argtypes = [i64, i64, vp, vp, vp, ctypes.POINTER(_Sizes)]
    lib.msq_plan.restype = ctypes.c_int
    lib.msq_quantize_pack.argtypes = [vp, ctypes.POINTER(_Weight), vp]
    lib.msq_quantize_pack.restype = ctypes.c_int
    lib.msq_gemm_workspace_bytes.argtypes = [i64, i64, i64]
    lib.msq_gemm_workspace_bytes.restype = sz
    lib.msq_gemm.argtypes = [vp, i64, ctypes.POINTER(_Weight), vp, vp, sz, vp]
    lib.msq_gemm.restype = ctypes.c_int
    lib.msq_gemm_ex.argtypes = [vp, i64, ctypes.POINTER(_Weight), vp, vp, sz,
                                ctypes.POINTER(_Options), vp]
    lib.msq_gemm_ex.restype = ctypes.c_int
    lib.msq_gemm_workspace_bytes_ex.argtypes = [i64, i64, i64, ctypes.POINTER(_Options)]
    lib.msq_gemm_workspace_bytes_ex.restype = sz
    lib.msq_gemm_group_workspace_bytes.argtypes = [i64, ctypes.POINTER(ctypes.POINTER(_Weight)),
                                                   ctypes.c_int]
    lib.msq_gemm_group_workspace_bytes.restype = sz
    lib.msq_gemm_group.argtypes = [ctypes.POINTER(vp), i64, ctypes.POINTER(ctypes.POINTER(_Weight)),
                                   ctypes.POINTER(vp), ctypes.c_int, vp, sz, vp]
    lib.msq_gemm_group.restype = ctypes.c_int
    lib.msq_gemm_group_workspace_bytes_ex.argtypes = [
        i64, ctypes.POINTER(ctypes.POINTER(_Weight)), ctypes.c_int, ctypes.POINTER(_Options)]
    lib.msq_gemm_group_workspace_bytes_ex.restype = sz
    lib.msq_gemm_group_ex.argtypes = [ctypes.POINTER(vp), i64,
                                      ctypes.POINTER(ctypes.POINTER(_Weight)), ctypes.POINTER(vp),
                                      ctypes.c_int, vp, sz, ctypes.POINTER(_Options), vp]
    lib.msq_gemm_group_ex.restype = ctypes.c_int
    lib.msq_alloc_workspace_bytes.argtypes = [i64]
    lib.msq_alloc_workspace_bytes.restype = sz
    lib.msq_allocate_bits.argtypes = [vp, i64, i64, vp, vp, sz, ctypes.POINTER(ctypes.c_int32), vp]
    lib.msq_allocate_bits.restype = ctypes.c_int
    lib.msq_reorder_workspace_bytes.argtypes = [i64, i64]
    lib.msq_reorder_workspace_bytes.restype = sz
    lib.msq_reorder_channels.argtypes = [vp, i64, i64, ctypes.c_int, vp, vp, vp, sz, vp]
    lib.msq_reorder_channels.restype = ctypes.c_int
    lib.msq_gemm_noalloc.argtypes = [vp, i64, ctypes.POINTER(_Weight), vp, vp]
    lib.msq_gemm_noalloc.restype = ctypes.c_int
    cache_p, seqs_p = ctypes.POINTER(_KvCache), ctypes.POINTER(_KvSeqs)
    attn_p = ctypes.POINTER(_KvAttn)
    lib.msq_kv_write.argtypes = [cache_p, seqs_p, vp, vp, i64, i64, vp, i64, i64, ctypes.c_int32,
                                 vp]
    lib.msq_kv_write.restype = ctypes.c_int
    lib.msq_kv_read.argtypes = [cache_p, seqs_p, vp, vp, vp, ctypes.c_int32, vp]
    lib.msq_kv_read.restype = ctypes.c_int
    lib.msq_kv_attention_plan.argtypes = [cache_p, seqs_p, attn_p, ctypes.POINTER(_KvPlan)]
    lib.msq_kv_attention_plan.restype = ctypes.c_int
    lib.msq_kv_attention_workspace_bytes.argtypes = [cache_p, seqs_p, attn_p]
    lib.msq_kv_attention_workspace_bytes.restype = sz
    lib.msq_kv_attention.argtypes = [cache_p, seqs_p, attn_p, vp, sz, vp]
    lib.msq_kv_attention.restype = ctypes.c_int
    lib.msq_status_string.argtypes = [ctypes.c_int]
    lib.msq_status_string.restype = ctypes.c_char_p
    lib.msq_format_version.argtypes = []
    lib.msq_format_version.restype = ctypes.c_int
    if lib.msq_format_version() != FORMAT_VERSION:
        raise OSError(f"{path} implements format {lib.msq_format_version()}, expected {FORMAT_VERSION}")
    _lib = lib
    return lib


def _check(status: int, where: str) -> None:
    if status != 0:
        raise MsqError(status, where)


def _host(a, dtype) -> np.ndarray:
    if hasattr(a, "detach"):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(a), dtype=dtype)


def plan(N: int, K: int, bits, perm_row, perm_col) -> dict:
    """Validate a problem on the host (no GPU needed) and return buffer sizes."""
    lib = load_library()
    b = _host(bits, np.uint8)
    pr = _host(perm_row, np.int32)
    pc = _host(perm_col, np.int32)
    if N > 0 and K > 0 and N % 64 == 0 and K % 128 == 0 and b.size != (N // 64) * (K // 128):
        raise ValueError("bits must have (N/64)*(K/128) entries")
    out = _Sizes()
    _check(lib.msq_plan(N, K, b.ctypes.data, pr.ctypes.data, pc.ctypes.data, ctypes.byref(out)),
           "msq_plan")
    return dict(code_bytes=out.code_bytes, scale_bytes=out.scale_bytes, zero_bytes=out.zero_bytes,
                offset_bytes=out.offset_bytes, blocks_per_bits=list(out.blocks_per_bits),
                mean_bits=out.mean_bits)


@functools.lru_cache(maxsize=None)
def _torch():
    import torch
    return torch


def _stream_handle(stream) -> int:
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _as_bf16_cuda(a, device):
    torch = _torch()
    if isinstance(a, np.ndarray):
        if a.dtype != np.uint16:
            raise TypeError("numpy inputs must be bf16 bit patterns (uint16)")
        a = torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16)
    if a.dtype in (torch.int16, torch.uint16):
        a = a.view(torch.bfloat16)
    if a.dtype != torch.bfloat16:
        raise TypeError(f"expected bf16 data, got {a.dtype}")
    return a.to(device).contiguous()


@dataclass
class PackedWeight:
    """Device buffers of one packed weight (format version 2).  Holds the tensors
    so their memory outlives every call that uses the descriptor."""
    N: int
    K: int
    bits: "object"          # uint8 [N/64][K/128]
    perm_row: "object"      # int32 [N]
    perm_col: "object"      # int32 [K]
    block_offset: "object"  # int32 view of uint32 [N/64][K/128]
    codes: "object"         # uint8 [code_bytes] (256-byte aligned by the allocator)
    scale: "object"         # float32 [N/64][K/128][64]
    zero: "object"          # uint8 [N/64][K/128][64]
    code_bytes: int
    mean_bits: float = 0.0
    tile16_blocks: int = 0

    def descriptor(self) -> _Weight:
        w = _Weight()
        w.N, w.K = self.N, self.K
        w.bits = self.bits.data_ptr()
        w.perm_row = self.perm_row.data_ptr()
        w.perm_col = self.perm_col.data_ptr()
        w.block_offset = self.block_offset.data_ptr()
        w.codes = self.codes.data_ptr() if self.code_bytes > 0 else None
        w.scale = self.scale.data_ptr()
        w.zero = self.zero.data_ptr()
        w.code_bytes = self.code_bytes
        w.tile16_blocks = self.tile16_blocks
        return w

    def to_numpy(self) -> dict:
        return dict(bits=self.bits.cpu().numpy(), perm_row=self.perm_row.cpu().numpy(),
                    perm_col=self.perm_col.cpu().numpy(),
                    block_offset=self.block_offset.cpu().numpy().view(np.uint32),
                    codes=self.codes.cpu().numpy()[: self.code_bytes],
                    scale=self.scale.cpu().numpy(), zero=self.zero.cpu().numpy())

    def clone(self) -> "PackedWeight":
        """Independent copy of every buffer (used to defeat caches in benchmarks)."""
        return PackedWeight(self.N, self.K, self.bits.clone(), self.perm_row.clone(),
                            self.perm_col.clone(), self.block_offset.clone(), self.codes.clone(),
                            self.scale.clone(), self.zero.clone(), self.code_bytes, self.mean_bits,
                            self.tile16_blocks)

    @property
    def packed_bytes(self) -> int:
        """Bytes the decode kernel must read for the weight: codes + scale/zero of live
        blocks + bit map and offsets + permutations."""
        nb = int(self.bits.numel())
        live = int((self.bits != 0).sum().item())
        return self.code_bytes + 320 * live + 5 * nb + 4 * (self.N + self.K)


def allocate_packed(N: int, K: int, bits, perm_row, perm_col, device="cuda") -> PackedWeight:
    """Validate the problem on the host (msq_plan, the one validation) and allocate the
    device buffers of its packed weight; the bit map and permutations are copied in."""
    torch = _torch()
    bh = _host(bits, np.uint8)
    if N % 64 == 0 and K % 128 == 0 and N > 0 and K > 0:
        bh = bh.reshape(N // 64, K // 128)
    ph = _host(perm_row, np.int32)
    qh = _host(perm_col, np.int32)
    sizes = plan(N, K, bh, ph, qh)
    dev = torch.device(device)
    code_bytes = int(sizes["code_bytes"])
    return PackedWeight(
        N, K,
        bits=torch.from_numpy(bh.copy()).to(dev),
        perm_row=torch.from_numpy(ph.copy()).to(dev),
        perm_col=torch.from_numpy(qh.copy()).to(dev),
        block_offset=torch.empty(bh.shape, dtype=torch.int32, device=dev),
        codes=torch.empty(max(code_bytes, 256), dtype=torch.uint8, device=dev),
        scale=torch.empty((N // 64, K // 128, 64), dtype=torch.float32, device=dev),
        zero=torch.empty((N // 64, K // 128, 64), dtype=torch.uint8, device=dev),
        code_bytes=code_bytes, mean_bits=float(sizes["mean_bits"]),
        tile16_blocks=int(sizes["blocks_per_bits"][16]))


def pack_into(W, pw: PackedWeight, stream=None) -> PackedWeight:
    """msq_quantize_pack of W (bf16 [N][K] on the weight's device) into the buffers of
    pw (from allocate_packed); asynchronous on the stream."""
    lib = load_library()
    Wd = _as_bf16_cuda(W, pw.bits.device)
    if tuple(Wd.shape) != (pw.N, pw.K):
        raise ValueError(f"W must be [{pw.N}][{pw.K}]")
    w = pw.descriptor()
    _check(lib.msq_quantize_pack(Wd.data_ptr(), ctypes.byref(w), _stream_handle(stream)),
           "msq_quantize_pack")
    return pw


def quantize_pack(W, bits, perm_row, perm_col, device="cuda", stream=None) -> PackedWeight:
    """Quantize and pack W (bf16 [N][K], original order) on the GPU."""
    Wd = _as_bf16_cuda(W, device)
    N, K = int(Wd.shape[0]), int(Wd.shape[1])
    pw = allocate_packed(N, K, bits, perm_row, perm_col, device=Wd.device)
    return pack_into(Wd, pw, stream=stream)


def pack_bytes(pw: PackedWeight) -> int:
    """HBM bytes the pack must move: W read (2 N K), permutations and bit map read,
    offsets, codes, scales and zero points written."""
    nb = int(pw.bits.numel())
    return (2 * pw.N * pw.K + 4 * (pw.N + pw.K) + nb + 4 * nb + pw.code_bytes
            + 4 * pw.N * (pw.K // 128) + pw.N * (pw.K // 128))


def workspace_bytes(M: int, N: int, K: int, kernel: str = "auto",
                    options: Optional[dict] = None) -> int:
    """Workspace of msq_gemm (automatic choices) or of msq_gemm_ex with these choices."""
    o = _options(kernel, options)
    lib = load_library()
    if o is None:
        return int(lib.msq_gemm_workspace_bytes(M, N, K))
    return int(lib.msq_gemm_workspace_bytes_ex(M, N, K, ctypes.byref(o)))


GROUP_MAX = 8


def _descriptor_array(pws):
    descs = [pw.descriptor() for pw in pws]
    arr = (ctypes.POINTER(_Weight) * len(descs))(*[ctypes.pointer(d) for d in descs])
    return descs, arr


def group_workspace_bytes(M: int, pws, options: Optional[dict] = None) -> int:
    descs, arr = _descriptor_array(pws)
    o = _options("auto", options)
    lib = load_library()
    if o is None:
        return int(lib.msq_gemm_group_workspace_bytes(M, arr, len(descs)))
    return int(lib.msq_gemm_group_workspace_bytes_ex(M, arr, len(descs), ctypes.byref(o)))


def gemm_group(xs, pws, outs=None, workspace=None, stream=None, options: Optional[dict] = None):
    """[x_i . W_i^T] for up to GROUP_MAX packed weights in one call (M == 1: one decode
    launch for all of them, plus one prep launch if some have several K ranges; M = 2..32:
    one gather and one decode launch; large M: one gather and one GEMM launch).  xs: one activation per weight (the same tensor may repeat); returns
    the list of fp32 [M][N_i] outputs."""
    torch = _torch()
    lib = load_library()
    pws = list(pws)
    if not 1 <= len(pws) <= GROUP_MAX or len(xs) != len(pws):
        raise ValueError(f"1 to {GROUP_MAX} weights, one activation each")
    xds = [_as_bf16_cuda(x, pw.bits.device) for x, pw in zip(xs, pws)]
    M = int(xds[0].shape[0])
    for xd, pw in zip(xds, pws):
        if xd.dim() != 2 or xd.shape[1] != pw.K or int(xd.shape[0]) != M:
            raise ValueError(f"each x must be [M][K] of its weight, one M for all")
    if outs is None:
        outs = [torch.empty((M, pw.N), dtype=torch.float32, device=xds[0].device) for pw in pws]
    descs, arr = _descriptor_array(pws)
    need = group_workspace_bytes(M, pws, options)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=xds[0].device)
    xa = (ctypes.c_void_p * len(xds))(*[xd.data_ptr() for xd in xds])
    ya = (ctypes.c_void_p * len(outs))(*[y.data_ptr() for y in outs])
    o = _options("auto", options)
    if M > 0:
        ws_ptr = workspace.data_ptr() if need > 0 else None
        if o is None:
            st = lib.msq_gemm_group(xa, M, arr, ya, len(descs), ws_ptr, workspace.numel(),
                                    _stream_handle(stream))
        else:
            st = lib.msq_gemm_group_ex(xa, M, arr, ya, len(descs), ws_ptr, workspace.numel(),
                                       ctypes.byref(o), _stream_handle(stream))
        _check(st, "msq_gemm_group")
    return outs


def gemm(x, pw: PackedWeight, kernel: str = "auto", out=None, workspace=None, stream=None,
         options: Optional[dict] = None):
    """y = x . W^T (fp32 [M][N], original row order) from packed weights.  kernel and
    options (keys gemv_split, gemv_waves, m1_prep, gemm_split) select the launch
    (msq_gemm_ex); the defaults are msq_gemm's automatic choices."""
    torch = _torch()
    lib = load_library()
    xd = _as_bf16_cuda(x, pw.bits.device)
    if xd.dim() != 2 or xd.shape[1] != pw.K:
        raise ValueError(f"x must be [M][{pw.K}]")
    M = int(xd.shape[0])
    if out is None:
        out = torch.empty((M, pw.N), dtype=torch.float32, device=xd.device)
    need = workspace_bytes(M, pw.N, pw.K, kernel, options)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=xd.device)
    w = pw.descriptor()
    ws_ptr = workspace.data_ptr() if need > 0 else None
    o = _options(kernel, options)
    xp = xd.data_ptr() if M > 0 else None
    yp = out.data_ptr() if M > 0 else None
    if o is None:
        st = lib.msq_gemm(xp, M, ctypes.byref(w), yp, ws_ptr, workspace.numel(),
                          _stream_handle(stream))
    else:
        st = lib.msq_gemm_ex(xp, M, ctypes.byref(w), yp, ws_ptr, workspace.numel(),
                             ctypes.byref(o), _stream_handle(stream))
    _check(st, "msq_gemm")
    return out


NOALLOC_SCRATCH_BYTES = 64 << 20


def gemm_noalloc(x, pw: PackedWeight, out=None, stream=None):
    """msq_gemm_noalloc: y = x . W^T with the library's own static device scratch as the
    workspace (no device allocation inside the call; out is allocated here if None)."""
    torch = _torch()
    lib = load_library()
    xd = _as_bf16_cuda(x, pw.bits.device)
    if xd.dim() != 2 or xd.shape[1] != pw.K:
        raise ValueError(f"x must be [M][{pw.K}]")
    M = int(xd.shape[0])
    if out is None:
        out = torch.empty((M, pw.N), dtype=torch.float32, device=xd.device)
    w = pw.descriptor()
    _check(lib.msq_gemm_noalloc(xd.data_ptr() if M > 0 else None, M, ctypes.byref(w),
                                out.data_ptr() if M > 0 else None, _stream_handle(stream)),
           "msq_gemm_noalloc")
    return out


ALLOC_LEVELS = (0, 1, 2, 3, 4, 8)


def alloc_workspace_bytes(n_blocks: int) -> int:
    return int(load_library().msq_alloc_workspace_bytes(int(n_blocks)))


def allocate_bits(utility, budget_bits: int, workspace=None, stream=None):
    """Bitwidth per block under a budget (msq_allocate_bits).  utility: fp32
    [n_blocks][6] for bitwidths ALLOC_LEVELS (numpy or torch).  Returns (bits as a
    uint8 device tensor [n_blocks], batched iterations)."""
    torch = _torch()
    lib = load_library()
    u = torch.as_tensor(utility)
    if u.dtype != torch.float32 or u.dim() != 2 or u.shape[1] != len(ALLOC_LEVELS):
        raise ValueError("utility must be float32 [n_blocks][6]")
    u = u.to("cuda").contiguous()
    n = int(u.shape[0])
    bits = torch.empty(n, dtype=torch.uint8, device=u.device)
    need = alloc_workspace_bytes(n)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=u.device)
    iters = ctypes.c_int32(0)
    _check(lib.msq_allocate_bits(u.data_ptr(), n, int(budget_bits), bits.data_ptr(),
                                 workspace.data_ptr(), workspace.numel(), ctypes.byref(iters),
                                 _stream_handle(stream)), "msq_allocate_bits")
    return bits, int(iters.value)


def reorder_channels(saliency, reorder_rows: bool = True, workspace=None, stream=None):
    """(perm_row, perm_col) as int32 device tensors from a saliency map fp32 [N][K]
    (msq_reorder_channels): rows and columns by total saliency, descending."""
    torch = _torch()
    lib = load_library()
    S = torch.as_tensor(saliency)
    if S.dtype != torch.float32 or S.dim() != 2:
        raise ValueError("saliency must be float32 [N][K]")
    S = S.to("cuda").contiguous()
    N, K = int(S.shape[0]), int(S.shape[1])
    pr = torch.empty(N, dtype=torch.int32, device=S.device)
    pc = torch.empty(K, dtype=torch.int32, device=S.device)
    need = int(lib.msq_reorder_workspace_bytes(N, K))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=S.device)
    _check(lib.msq_reorder_channels(S.data_ptr(), N, K, int(bool(reorder_rows)), pr.data_ptr(),
                                    pc.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                    _stream_handle(stream)), "msq_reorder_channels")
    return pr, pc


# ---- 8-bit key/value cache ---------------------------------------------------------
KV_HEAD_DIMS = (64, 128, 256)
KV_BLOCK_TOKENS = (32, 64, 128, 256)


@dataclass
class KVCache:
    """Device buffers of an 8-bit key/value cache: blocks of block_tokens tokens, one fp32
    scale per block and head (layout and quantiser: include/msq.h).  Block tables say which
    blocks a sequence has; handing blocks out is the caller's.  Fields may be set anew (a
    cache that grows or moves): the next call checks and uses them."""
    num_blocks: int
    kv_heads: int
    head_dim: int
    block_tokens: int
    k_codes: "object"   # uint8 [num_blocks][kv_heads][block_tokens * head_dim]
    v_codes: "object"
    k_scale: "object"   # float32 [num_blocks][kv_heads]
    v_scale: "object"

    def __post_init__(self):
        self.descriptor()

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name in _KV_CACHE_FIELDS:
            object.__setattr__(self, "_desc", None)

    def descriptor(self) -> _KvCache:
        if self._desc is None:
            torch = _torch()
            scales = self.num_blocks * self.kv_heads
            sizes = {"k_codes": scales * self.block_tokens * self.head_dim, "k_scale": scales}
            index = self.k_codes.get_device()
            for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
                t, codes = getattr(self, name), name.endswith("codes")
                want, numel = (torch.uint8, sizes["k_codes"]) if codes else (torch.float32, sizes["k_scale"])
                if t.dtype is not want or t.numel() != numel or not t.is_contiguous() or \
                        t.get_device() != index or t.device.type != self.k_codes.device.type:
                    raise ValueError(f"{name} must be contiguous {want} of {numel} values, on the "
                                     "device of the other buffers")
            d = _KvCache()
            _pack(_KV_CACHE, d, "the cache's sizes", self.num_blocks, self.kv_heads, self.head_dim,
                  self.block_tokens, self.k_codes.data_ptr(), self.v_codes.data_ptr(),
                  self.k_scale.data_ptr(), self.v_scale.data_ptr())
            self._index = index
            self._desc = d
        return self._desc

    @property
    def device(self):
        return self.k_codes.device

    @property
    def nbytes(self) -> int:
        """Device bytes of the codes and scales."""
        return 2 * int(self.k_codes.numel()) + 8 * int(self.k_scale.numel())


def allocate_kv_cache(num_blocks: int, kv_heads: int, head_dim: int, block_tokens: int = 64,
                      device="cuda") -> KVCache:
    """An empty cache.  head_dim from KV_HEAD_DIMS, block_tokens from KV_BLOCK_TOKENS.  Codes
    start undefined (no call uses slots that were never written); scales start at 0."""
    torch = _torch()
    if head_dim not in KV_HEAD_DIMS or block_tokens not in KV_BLOCK_TOKENS:
        raise ValueError(f"head_dim must be one of {KV_HEAD_DIMS}, block_tokens of {KV_BLOCK_TOKENS}")
    if num_blocks < 1 or kv_heads < 1:
        raise ValueError("num_blocks and kv_heads must be positive")
    dev = torch.device(device)
    codes = [torch.empty((num_blocks, kv_heads, block_tokens * head_dim), dtype=torch.uint8,
                         device=dev) for _ in range(2)]
    scale = [torch.zeros((num_blocks, kv_heads), dtype=torch.float32, device=dev) for _ in range(2)]
    return KVCache(num_blocks, kv_heads, head_dim, block_tokens, *codes, *scale)


_KV_DTYPE: dict = {}


def _kv_dtype(dtype) -> int:
    code = _KV_DTYPE.get(dtype)
    if code is None:
        torch = _torch()
        _KV_DTYPE.update({torch.bfloat16: 0, torch.float32: 1})
        if dtype not in _KV_DTYPE:
            raise TypeError(f"expected bfloat16 or float32, got {dtype}")
        code = _KV_DTYPE[dtype]
    return code


def _kv_rows(t, name, heads, dim, index):
    """t as (tensor, rows, address, token stride, head stride, type) of [rows][heads][dim] the
    kernels can read: any token and head strides that are multiples of 16 bytes with contiguous
    dims; anything else is copied."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [rows][{heads}][{dim}]")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on the cache's device")
    code = _KV_DTYPE.get(t.dtype)
    if code is None:
        code = _kv_dtype(t.dtype)
    st, sh, sd = t.stride()
    at = t.data_ptr()
    per16 = 4 if code else 8
    if sd != 1 or st % per16 or sh % per16 or at % 16:
        t = t.clone(memory_format=_torch().contiguous_format)
        at, st, sh = t.data_ptr(), heads * dim, dim
    return t, shape[0], at, st, sh, code


def _kv_seqs_struct(batch, width, table, offset, total, max_count) -> _KvSeqs:
    s = _KvSeqs()
    try:
        _KV_SEQS.pack_into(s, 0, batch, width, table, offset, total, max_count)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"rows, max_count or block_table: {e}") from None
    return s


def _kv_index(t, name, count, index):
    """t as a contiguous int32 tensor of count entries on the cache's device."""
    if t.dtype is not _torch().int32 or t.dim() != 1 or t.numel() != count or t.get_device() != index:
        raise ValueError(f"{name} must be int32 [{count}] on the cache's device")
    return t if t.is_contiguous() else t.contiguous()


def _kv_seqs(cache: KVCache, block_table, offset, total: int, max_count: int):
    """(sequences struct, the tensors it points into)."""
    shape = block_table.shape
    if len(shape) != 2 or shape[1] < 1 or block_table.dtype is not _torch().int32 or \
            block_table.get_device() != cache._index:
        raise ValueError("block_table must be int32 [batch][entries] on the cache's device")
    batch, width = shape
    if not block_table.is_contiguous():
        block_table = block_table.contiguous()
    if offset is None:
        if total % max(batch, 1) or (batch == 0 and total):
            raise ValueError("without offset every sequence has the same number of rows")
        return _kv_seqs_struct(batch, width, block_table.data_ptr(), 0, total, max_count), block_table
    offset = _kv_index(offset, "offset", batch + 1, cache._index)
    return (_kv_seqs_struct(batch, width, block_table.data_ptr(), offset.data_ptr(), total, max_count),
            (block_table, offset))


def _kv_on(cache: KVCache, stream, tensors, call):
    """call() with the cache's device and the given stream current, so that what it allocates
    belongs to that stream; the tensors it was given are marked as used there."""
    torch = _torch()
    if cache._index < 0:
        raise ValueError(f"the cache is on {cache.device}: its operators run on a GPU")
    if stream is not None and stream.device_index != cache._index:
        raise ValueError(f"the stream is on device {stream.device_index}, the cache on {cache.device}")
    with torch.cuda.device(cache._index):
        with torch.cuda.stream(torch.cuda.current_stream() if stream is None else stream) as _:
            used = torch.cuda.current_stream()
            result = call()
    for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale, *tensors):
        if t is not None and t.is_cuda:
            t.record_stream(used)
    return result


def kv_write(cache: KVCache, k, v, block_table, first, offset=None, max_count: int = 0,
             stream=None) -> None:
    """Quantise new tokens' keys and values into the cache (msq_kv_write).

    k, v: [rows][kv_heads][head_dim] bf16 or fp32 (one type for both).  block_table: int32
    [batch][entries].  first: int32 [batch], the position of each sequence's first new token,
    which is the number of tokens it has in the cache (negative: leave the sequence out).
    offset: int32 [batch + 1], sequence b's rows are offset[b] .. offset[b + 1] - 1; None:
    rows / batch each.  max_count: the largest sequence's rows, if known (else all rows)."""
    desc = cache._desc or cache.descriptor()
    index, cuda = cache._index, _torch()._C
    if stream is not None or index < 0 or cuda._cuda_getDevice() != index:
        return _kv_on(cache, stream, (k, v, block_table, first, offset),
                      lambda: kv_write(cache, k, v, block_table, first, offset, max_count))
    heads, dim = cache.kv_heads, cache.head_dim
    k, rows, k_at, k_st, k_sh, code = _kv_rows(k, "k", heads, dim, index)
    v, v_rows, v_at, v_st, v_sh, v_code = _kv_rows(v, "v", heads, dim, index)
    if v_rows != rows or v_code != code:
        raise ValueError("k and v must have the same rows and type")
    s, keep = _kv_seqs(cache, block_table, offset, rows, max_count)
    first = _kv_index(first, "first", s.batch, index)
    status = load_library().msq_kv_write(desc, s, first.data_ptr(), k_at, k_st, k_sh, v_at,
                                         v_st, v_sh, code, cuda._cuda_getCurrentRawStream(index))
    if status:
        raise MsqError(status, "msq_kv_write")


def kv_read(cache: KVCache, block_table, first, offset=None, total: Optional[int] = None,
            max_count: int = 0, dtype=None, stream=None):
    """Read positions first[b] .. first[b] + rows - 1 of every sequence back (msq_kv_read):
    (k, v), [total][kv_heads][head_dim] of dtype (bf16 unless given; or fp32), code * scale.
    offset as in kv_write, total its last entry; with offset None, total / batch rows each."""
    desc = cache._desc or cache.descriptor()
    index, cuda = cache._index, _torch()._C
    if stream is not None or index < 0 or cuda._cuda_getDevice() != index:
        return _kv_on(cache, stream, (block_table, first, offset),
                      lambda: kv_read(cache, block_table, first, offset, total, max_count, dtype))
    torch = _torch()
    if total is None or total < 0:
        raise ValueError("total: the number of rows to read")
    s, keep = _kv_seqs(cache, block_table, offset, total, max_count)
    first = _kv_index(first, "first", s.batch, index)
    dtype = dtype or torch.bfloat16
    code = _kv_dtype(dtype)
    k = torch.empty((total, cache.kv_heads, cache.head_dim), dtype=dtype, device=cache.device)
    v = torch.empty_like(k)
    status = load_library().msq_kv_read(desc, s, first.data_ptr(), k.data_ptr(),
                                        v.data_ptr(), code, cuda._cuda_getCurrentRawStream(index))
    if status:
        raise MsqError(status, "msq_kv_read")
    return k, v


def _kv_sizes(rows, q_heads, batch, entries, max_count, max_kv_len, causal, window, ragged):
    """What the size queries look at; of an offset only whether it is there."""
    a = _KvAttn()
    _pack(_KV_ATTN, a, "q_heads, max_kv_len or window", 0, 0, 0, 0, q_heads, 0, max_kv_len, 0.0,
          1 if causal else 0, window, 0, 0, 0)
    return _kv_seqs_struct(batch, entries, 0, 1 if ragged else 0, rows, max_count), a


def kv_attention_workspace_bytes(cache: KVCache, rows: int, q_heads: int, batch: int,
                                 max_count: int, max_kv_len: int, causal: bool = True,
                                 window: int = 0) -> int:
    """Workspace of kv_attention for calls of these sizes (rows: query rows of all sequences)
    whose block tables have no more entries than max_kv_len tokens need, whatever max_kv_len they
    are given.  Fewer sequences can need more, since theirs are split further: a buffer for calls
    of several batches takes the largest."""
    width = max(1, -(-max_kv_len // cache.block_tokens))  # the table's length stands for max_kv_len
    s, a = _kv_sizes(rows, q_heads, batch, width, max_count, 0, causal, window, True)
    desc = cache._desc or cache.descriptor()
    return int(load_library().msq_kv_attention_workspace_bytes(desc, s, a))


def kv_attention_plan(cache: KVCache, rows: int, q_heads: int, batch: int, table_entries: int,
                      max_count: int = 0, max_kv_len: int = 0, causal: bool = True, window: int = 0,
                      ragged: bool = True) -> dict:
    """How kv_attention runs a call of these sizes (msq_kv_attention_plan): tile_rows and
    wavefronts of its kernel's workgroups, the parts that a tile's tokens are split into, join
    ("none", "inside" the launch or by a "launch" of its own) and workspace_bytes.  Arguments as
    of kv_attention; ragged: whether it is given an offset."""
    s, a = _kv_sizes(rows, q_heads, batch, table_entries, max_count, max_kv_len, causal, window, ragged)
    plan = _KvPlan()
    _check(load_library().msq_kv_attention_plan(cache._desc or cache.descriptor(), s, a, plan),
           "msq_kv_attention_plan")
    return dict(tile_rows=plan.tile_rows, wavefronts=plan.wavefronts, parts=plan.parts,
                join=("none", "inside", "launch")[plan.join], workspace_bytes=plan.workspace_bytes)


def kv_attention(q, cache: KVCache, block_table, kv_len, offset=None, max_count: int = 0,
                 max_kv_len: int = 0, scale: float = 0.0, causal: bool = True, window: int = 0,
                 out=None, out_dtype=None, return_lse: bool = False, workspace=None, stream=None):
    """Attention of new tokens' queries over the cache (msq_kv_attention).

    q: [rows][q_heads][head_dim] bf16 or fp32, q_heads a multiple of kv_heads.  kv_len: int32
    [batch], the tokens each sequence has in the cache, the queries' own among them: with
    causal, query i of n stands at position kv_len - n + i and sees positions up to its own,
    the last `window` of them if window > 0.  offset, max_count as in kv_write.  max_kv_len:
    about the largest kv_len, for the split of the work (0: the block table's length).
    scale: of the scores (0: 1 / sqrt(head_dim)).  Returns out [rows][q_heads][head_dim] (bf16
    unless out or out_dtype says fp32), with return_lse also the fp32 [rows][q_heads] natural
    log of each row's softmax denominator.  A query that sees nothing gives zeros and -inf; rows
    outside every sequence are not written.  Products are of f16 operands, the softmax weights
    among them (some 2^-12 of the values' size in fp32 results); fp32 queries count by 22 bits
    for fp32 results, by 11 for bf16 ones (include/msq.h).  workspace: uint8 tensor to reuse, of kv_attention_workspace_bytes."""
    desc = cache._desc or cache.descriptor()
    index, cuda = cache._index, _torch()._C
    if stream is not None or index < 0 or cuda._cuda_getDevice() != index:
        return _kv_on(cache, stream, (q, block_table, kv_len, offset, out, workspace),
                      lambda: kv_attention(q, cache, block_table, kv_len, offset, max_count,
                                           max_kv_len, scale, causal, window, out, out_dtype,
                                           return_lse, workspace))
    torch = _torch()
    lib = load_library()
    if q.dim() != 3:
        raise ValueError("q must be [rows][q_heads][head_dim]")
    heads, dim = q.size(1), cache.head_dim
    q, rows, q_at, q_st, q_sh, q_code = _kv_rows(q, "q", heads, dim, index)
    s, keep = _kv_seqs(cache, block_table, offset, rows, max_count)
    kv_len = _kv_index(kv_len, "kv_len", s.batch, index)
    if out is None:
        out = torch.empty_like(q, dtype=out_dtype or torch.bfloat16,
                               memory_format=torch.contiguous_format)
    elif out.shape != (rows, heads, dim) or not out.is_contiguous() or out.get_device() != index or \
            (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out must be contiguous, [rows][q_heads][head_dim], on the cache's device")
    lse = torch.empty((rows, heads), dtype=torch.float32, device=cache.device) if return_lse else None
    a = _KvAttn()
    try:
        _KV_ATTN.pack_into(a, 0, q_at, q_st, q_sh, q_code, heads, kv_len.data_ptr(), max_kv_len,
                           scale, 1 if causal else 0, window, out.data_ptr(), _kv_dtype(out.dtype),
                           0 if lse is None else lse.data_ptr())
    except (struct.error, OverflowError) as e:
        raise ValueError(f"max_kv_len, scale or window: {e}") from None
    if workspace is None:
        need = int(lib.msq_kv_attention_workspace_bytes(desc, s, a))
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=cache.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous, on the cache's device")
    status = lib.msq_kv_attention(desc, s, a, workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(),
                                  cuda._cuda_getCurrentRawStream(index))
    if status:
        raise MsqError(status, "msq_kv_attention")
    return (out, lse) if return_lse else out
