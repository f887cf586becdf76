"""Thin Python binding over the C ABI in include/bitnet_tm.h.

Argument marshalling only: every step of the projection runs in the gfx950 HIP
kernels of ``libbitnet_tm.so``.  torch supplies device memory and the current
stream; no torch type crosses the ABI.  If the library is missing or the device
is not a gfx950, calls raise -- there is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

from . import _build

LIB_PATH = _build.LIB_PATH

BITNET_OK = 0
BITNET_MAX_GROUP = 256
UNIT = 128

_c = ctypes
_p = _c.c_void_p
_i64 = _c.c_int64
_i32 = _c.c_int32
_sz = _c.c_size_t


class BitnetError(RuntimeError):
    def __init__(self, status: int, fn: str):
        self.status = status
        super().__init__(f"{fn}: status {status} ({status_string(status)})")


class bitnet_problem(ctypes.Structure):
    _fields_ = [("x", _p), ("packed", _p), ("w_scale", _p), ("y", _p),
                ("N", _i64), ("K", _i64)]


class bitnet_kv_cache(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("k_scale", _p), ("v_scale", _p),
                ("layer_stride", _i64), ("page_stride", _i64), ("head_stride", _i64),
                ("token_stride", _i64), ("dtype", _i32), ("layers", _i32), ("pages", _i32),
                ("kv_heads", _i32), ("page_size", _i32), ("head_dim", _i32)]


class bitnet_kv_pool(ctypes.Structure):
    _fields_ = [("tables", _p), ("owned", _p), ("free_pages", _p), ("rows", _i32),
                ("max_pages", _i32), ("pages", _i32), ("page_size", _i32)]


EXPORTS = (
    "bitnet_status_string", "bitnet_packed_bytes", "bitnet_ternarize_workspace_bytes",
    "bitnet_ternarize_pack", "bitnet_quant_act", "bitnet_matmul_workspace_bytes",
    "bitnet_ternary_matmul", "bitnet_ternary_matmul_q8", "bitnet_grouped_workspace_bytes",
    "bitnet_ternary_matmul_grouped", "bitnet_stages_workspace_bytes",
    "bitnet_ternary_matmul_stages", "bitnet_ternary_matmul_lut_grouped",
    "bitnet_i8_quant_workspace_bytes", "bitnet_i8_quant_weights",
    "bitnet_i8_linear_workspace_bytes", "bitnet_i8_linear",
)

_lib = None


def lib():
    """Load libbitnet_tm.so (after torch, so both share one HIP runtime)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"HIP library {LIB_PATH} is not built; run __graft_entry__.build() "
                "(python -m ternary_weight_decoder_amd._build)")
        L = ctypes.CDLL(LIB_PATH)
        L.bitnet_status_string.argtypes = [_i32]
        L.bitnet_status_string.restype = _c.c_char_p
        L.bitnet_packed_bytes.argtypes = [_i64, _i64]
        L.bitnet_packed_bytes.restype = _sz
        L.bitnet_ternarize_workspace_bytes.argtypes = [_i64]
        L.bitnet_ternarize_workspace_bytes.restype = _sz
        L.bitnet_ternarize_pack.argtypes = [_p, _i64, _i64, _p, _p, _p, _sz, _p]
        L.bitnet_ternarize_pack.restype = _i32
        L.bitnet_quant_act.argtypes = [_p, _i64, _i64, _p, _p, _p]
        L.bitnet_quant_act.restype = _i32
        L.bitnet_matmul_workspace_bytes.argtypes = [_i64, _i64]
        L.bitnet_matmul_workspace_bytes.restype = _sz
        L.bitnet_ternary_matmul.argtypes = [_i64, _i64, _i64, _p, _p, _p, _p, _p, _sz, _p, _p,
                                            _p, _p]
        L.bitnet_ternary_matmul.restype = _i32
        L.bitnet_ternary_matmul_q8.argtypes = [_i64, _i64, _i64, _p, _p, _p, _p, _p, _p, _sz,
                                               _p, _p]
        L.bitnet_ternary_matmul_q8.restype = _i32
        L.bitnet_grouped_workspace_bytes.argtypes = [_i64, _p, _i32]
        L.bitnet_grouped_workspace_bytes.restype = _sz
        L.bitnet_ternary_matmul_grouped.argtypes = [_i64, _p, _i32, _p, _p, _sz, _p]
        L.bitnet_ternary_matmul_grouped.restype = _i32
        L.bitnet_stages_workspace_bytes.argtypes = [_i64, _p, _i32]
        L.bitnet_stages_workspace_bytes.restype = _sz
        L.bitnet_ternary_matmul_stages.argtypes = [_i64, _p, _i32, _p, _i32, _p, _p, _sz, _p]
        L.bitnet_ternary_matmul_stages.restype = _i32
        L.bitnet_ternary_matmul_lut_grouped.argtypes = [_p, _i32, _p, _p]
        L.bitnet_ternary_matmul_lut_grouped.restype = _i32
        L.bitnet_i8_quant_workspace_bytes.argtypes = []
        L.bitnet_i8_quant_workspace_bytes.restype = _sz
        L.bitnet_i8_quant_weights.argtypes = [_p, _i64, _i64, _p, _p, _p, _sz, _p]
        L.bitnet_i8_quant_weights.restype = _i32
        L.bitnet_i8_linear_workspace_bytes.argtypes = [_i64, _i64]
        L.bitnet_i8_linear_workspace_bytes.restype = _sz
        L.bitnet_i8_linear.argtypes = [_i64, _i64, _i64, _p, _p, _p, _p, _i32, _p, _p, _sz, _p,
                                       _p]
        L.bitnet_i8_linear.restype = _i32
        L.bitnet_scratch_bytes.argtypes = []
        L.bitnet_scratch_bytes.restype = _sz
        L.bitnet_ternary_matmul_noalloc.argtypes = [_i64, _i64, _i64, _p, _p, _p, _p, _p, _p,
                                                    _p, _p]
        L.bitnet_ternary_matmul_noalloc.restype = _i32
        L.bitnet_i8_linear_rows.argtypes = [_i64, _i64, _i64, _p, _p, _p, _p, _i32, _p, _p, _sz,
                                            _p, _p]
        L.bitnet_i8_linear_rows.restype = _i32
        L.bitnet_ternary_matmul_grouped_overlap.argtypes = [_i64, _p, _i32, _p, _i32, _p, _sz, _p,
                                                            _p]
        L.bitnet_ternary_matmul_grouped_overlap.restype = _i32
        L.bitnet_i8_dwconv_quant_weights.argtypes = [_p, _i64, _i64, _p, _p, _p]
        L.bitnet_i8_dwconv_quant_weights.restype = _i32
        L.bitnet_i8_dwconv_workspace_bytes.argtypes = [_i64, _i64, _i64]
        L.bitnet_i8_dwconv_workspace_bytes.restype = _sz
        L.bitnet_i8_dwconv.argtypes = [_i64, _i64, _i64, _i64, _p, _p, _p, _p, _i32, _p, _p, _sz,
                                       _p, _p, _p]
        L.bitnet_i8_dwconv.restype = _i32
        L.bitnet_table_bytes.argtypes = [_i64, _i64]
        L.bitnet_table_bytes.restype = _sz
        L.bitnet_table_quant.argtypes = [_p, _i64, _i64, _p, _p, _p]
        L.bitnet_table_quant.restype = _i32
        L.bitnet_i8_quant_weights_rows.argtypes = [_p, _i64, _i64, _p, _p, _p]
        L.bitnet_i8_quant_weights_rows.restype = _i32
        L.bitnet_embed_lookup.argtypes = [_p, _i64, _p, _p, _i64, _i64, _p, _p]
        L.bitnet_embed_lookup.restype = _i32
        L.bitnet_lm_head.argtypes = [_i64, _i64, _i64, _p, _p, _p, _p, _p, _p, _p, _p]
        L.bitnet_lm_head.restype = _i32
        L.bitnet_kv_map.argtypes = [_p, _i64, _p, _p, _p, _p, _p, _p, _p, _p, _p]
        L.bitnet_kv_map.restype = _i32
        L.bitnet_kv_append.argtypes = [_p, _i32, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _p, _p,
                                       _i64, _p, _i64, _p, _p]
        L.bitnet_kv_append.restype = _i32
        L.bitnet_paged_attention_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, _i64]
        L.bitnet_paged_attention_workspace_bytes.restype = _sz
        L.bitnet_paged_attention.argtypes = [_p, _i32, _i64, _i64, _p, _i64, _p, _i64, _i64, _p,
                                             _p, _i64, _c.c_float, _p, _p, _p, _sz, _p]
        L.bitnet_paged_attention.restype = _i32
        L.bitnet_beam_select_workspace_bytes.argtypes = [_i64, _i64, _i64]
        L.bitnet_beam_select_workspace_bytes.restype = _sz
        L.bitnet_beam_select.argtypes = [_i64, _i64, _i64, _p, _i64, _p, _p, _i32, _p, _p, _p, _p,
                                         _p, _sz, _p]
        L.bitnet_beam_select.restype = _i32
        L.bitnet_beam_reorder.argtypes = [_p, _i64, _i64, _p, _p, _p, _p, _i64, _p]
        L.bitnet_beam_reorder.restype = _i32
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().bitnet_status_string(int(status)).decode()


def _check(status: int, fn: str) -> None:
    if status != BITNET_OK:
        raise BitnetError(status, fn)


def _ptr(t):   # (an int: every function's argtypes are declared)
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    # (torch.cuda.current_stream() builds an object: 2.7 us a call against 0.4.)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _dev(t: torch.Tensor, dtype, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ---------------------------------------------------------------------------
# Raw entry points: same names and arguments as the C ABI (tensors stand in for
# device pointers).  They allocate nothing.
# ---------------------------------------------------------------------------

def bitnet_packed_bytes(N: int, K: int) -> int:
    return int(lib().bitnet_packed_bytes(N, K))


def bitnet_ternarize_workspace_bytes(N: int) -> int:
    return int(lib().bitnet_ternarize_workspace_bytes(N))


def bitnet_matmul_workspace_bytes(M: int, K: int) -> int:
    return int(lib().bitnet_matmul_workspace_bytes(M, K))


def bitnet_ternarize_pack_into(W, N, K, packed, w_scale, workspace, stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().bitnet_ternarize_pack(_ptr(W), N, K, _ptr(packed), _ptr(w_scale),
                                       _ptr(workspace), ws_bytes, _stream(stream)),
           "bitnet_ternarize_pack")


def bitnet_quant_act_into(x, M, K, xq, x_scale, stream=None) -> None:
    _check(lib().bitnet_quant_act(_ptr(x), M, K, _ptr(xq), _ptr(x_scale), _stream(stream)),
           "bitnet_quant_act")


def bitnet_ternary_matmul_into(M, N, K, x, packed, w_scale, y, workspace, xq_out=None,
                               x_scale_out=None, acc_out=None, stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().bitnet_ternary_matmul(M, N, K, _ptr(x), _ptr(packed), _ptr(w_scale), _ptr(y),
                                       _ptr(workspace), ws_bytes, _ptr(xq_out),
                                       _ptr(x_scale_out), _ptr(acc_out), _stream(stream)),
           "bitnet_ternary_matmul")


def bitnet_ternary_matmul_q8_into(M, N, K, xq, x_scale, packed, w_scale, y, workspace,
                                  acc_out=None, stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().bitnet_ternary_matmul_q8(M, N, K, _ptr(xq), _ptr(x_scale), _ptr(packed),
                                          _ptr(w_scale), _ptr(y), _ptr(workspace), ws_bytes,
                                          _ptr(acc_out), _stream(stream)),
           "bitnet_ternary_matmul_q8")


# ---------------------------------------------------------------------------
# Convenience forms that allocate their outputs with torch (plumbing only).
# ---------------------------------------------------------------------------

def bitnet_scratch_bytes() -> int:
    return int(lib().bitnet_scratch_bytes())


def bitnet_ternary_matmul_noalloc_into(M, N, K, x, packed, w_scale, y, xq_out=None,
                                       x_scale_out=None, acc_out=None, stream=None) -> None:
    """The projection with the library's built-in scratch instead of a workspace."""
    _check(lib().bitnet_ternary_matmul_noalloc(M, N, K, _ptr(x), _ptr(packed), _ptr(w_scale),
                                               _ptr(y), _ptr(xq_out), _ptr(x_scale_out),
                                               _ptr(acc_out), _stream(stream)),
           "bitnet_ternary_matmul_noalloc")


def bitnet_ternarize_pack(W: torch.Tensor, stream=None):
    """fp32 W [N,K] -> (packed uint8 [N*K/4], w_scale fp32 [1]) on W's device."""
    _dev(W, torch.float32, "W")
    N, K = W.shape
    packed = torch.empty(max(N * K // 4, 1), dtype=torch.uint8, device=W.device)
    w_scale = torch.empty(1, dtype=torch.float32, device=W.device)
    ws = torch.empty(max(bitnet_ternarize_workspace_bytes(N), 16), dtype=torch.uint8,
                     device=W.device)
    bitnet_ternarize_pack_into(W, N, K, packed, w_scale, ws, stream)
    return packed, w_scale


def bitnet_quant_act(x: torch.Tensor, stream=None):
    """fp32 x [M,K] -> (xq int8 [M,K], x_scale fp32 [M])."""
    _dev(x, torch.float32, "x")
    M, K = x.shape
    xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    xs = torch.empty(M, dtype=torch.float32, device=x.device)
    bitnet_quant_act_into(x, M, K, xq, xs, stream)
    return xq, xs


def bitnet_ternary_matmul(x: torch.Tensor, packed: torch.Tensor, w_scale: torch.Tensor,
                          N: int, *, return_parts: bool = False, stream=None):
    """y [M,N] fp32; with return_parts also xq, x_scale and the int32 accumulators."""
    _dev(x, torch.float32, "x")
    _dev(packed, torch.uint8, "packed")
    _dev(w_scale, torch.float32, "w_scale")
    M, K = x.shape
    y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    ws = torch.empty(bitnet_matmul_workspace_bytes(M, K), dtype=torch.uint8, device=x.device)
    if return_parts:
        xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
        xs = torch.empty(M, dtype=torch.float32, device=x.device)
        acc = torch.empty((M, N), dtype=torch.int32, device=x.device)
        bitnet_ternary_matmul_into(M, N, K, x, packed, w_scale, y, ws, xq, xs, acc, stream)
        return {"y": y, "xq": xq, "x_scale": xs, "acc": acc}
    bitnet_ternary_matmul_into(M, N, K, x, packed, w_scale, y, ws, stream=stream)
    return y


def bitnet_ternary_matmul_q8(xq: torch.Tensor, x_scale: torch.Tensor, packed: torch.Tensor,
                             w_scale: torch.Tensor, N: int, *, return_acc: bool = False,
                             stream=None):
    _dev(xq, torch.int8, "xq")
    M, K = xq.shape
    y = torch.empty((M, N), dtype=torch.float32, device=xq.device)
    ws = torch.empty(bitnet_matmul_workspace_bytes(M, K), dtype=torch.uint8, device=xq.device)
    acc = torch.empty((M, N), dtype=torch.int32, device=xq.device) if return_acc else None
    bitnet_ternary_matmul_q8_into(M, N, K, xq, x_scale, packed, w_scale, y, ws, acc, stream)
    return (y, acc) if return_acc else y


class GroupedPlan:
    """A fixed set of independent projections with the same M, launched together.

    Holds the host and device copies of the problem array and the workspace, so
    that run() is a single C call with no allocation.
    """

    def __init__(self, M: int, xs, packeds, w_scales, ys, Ns, Ks, device=None):
        count = len(xs)
        if not 1 <= count <= BITNET_MAX_GROUP:
            raise ValueError(f"group size must be 1..{BITNET_MAX_GROUP}")
        self.M = int(M)
        self.count = count
        arr = (bitnet_problem * count)()
        for i in range(count):
            arr[i] = bitnet_problem(xs[i].data_ptr(), packeds[i].data_ptr(),
                                    w_scales[i].data_ptr(), ys[i].data_ptr(), int(Ns[i]),
                                    int(Ks[i]))
        self._keep = (list(xs), list(packeds), list(w_scales), list(ys))
        self.host = arr
        dev = device if device is not None else xs[0].device
        raw = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8)
        self.dev = raw.to(dev)
        nbytes = int(lib().bitnet_grouped_workspace_bytes(self.M, _c.byref(arr), count))
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
        self.ws_bytes = nbytes

    def run(self, stream=None) -> None:
        bitnet_ternary_matmul_grouped(self.M, self.dev, self.count, self.host, self.workspace,
                                      stream)

    def run_overlap(self, aux_stream, nchunks: int, stream=None) -> None:
        """The same call with the quantization of later chunks on aux_stream,
        overlapping the contraction of earlier ones (prefill, M > 16)."""
        bitnet_ternary_matmul_grouped_overlap(self.M, self.dev, self.count, self.host, nchunks,
                                              self.workspace, stream, aux_stream)


def bitnet_ternary_matmul_grouped_overlap(M, problems_dev, count, problems_host, nchunks,
                                          workspace, stream=None, aux_stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().bitnet_ternary_matmul_grouped_overlap(M, _ptr(problems_dev), count,
                                                       _c.byref(problems_host), int(nchunks),
                                                       _ptr(workspace), ws_bytes,
                                                       _stream(stream), _stream(aux_stream)),
           "bitnet_ternary_matmul_grouped_overlap")


def bitnet_grouped_workspace_bytes(M: int, problems_host, count: int) -> int:
    return int(lib().bitnet_grouped_workspace_bytes(M, _c.byref(problems_host), count))


def bitnet_ternary_matmul_grouped(M, problems_dev, count, problems_host, workspace,
                                  stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().bitnet_ternary_matmul_grouped(M, _ptr(problems_dev), count,
                                               _c.byref(problems_host), _ptr(workspace),
                                               ws_bytes, _stream(stream)),
           "bitnet_ternary_matmul_grouped")


def bitnet_i8_quant_weights_into(W, N, K, q, w_scale, workspace, stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().bitnet_i8_quant_weights(_ptr(W), N, K, _ptr(q), _ptr(w_scale), _ptr(workspace),
                                         ws_bytes, _stream(stream)),
           "bitnet_i8_quant_weights")


def bitnet_i8_quant_weights(W: torch.Tensor, stream=None):
    """fp32 W [N,K] -> (q int8 [N,K], w_scale fp32 [1]) on W's device (I8_S)."""
    _dev(W, torch.float32, "W")
    N, K = W.shape
    q = torch.empty((N, K), dtype=torch.int8, device=W.device)
    w_scale = torch.empty(1, dtype=torch.float32, device=W.device)
    ws = torch.empty(int(lib().bitnet_i8_quant_workspace_bytes()), dtype=torch.uint8,
                     device=W.device)
    bitnet_i8_quant_weights_into(W, N, K, q, w_scale, ws, stream)
    return q, w_scale


def bitnet_i8_linear_workspace_bytes(M: int, K: int) -> int:
    return int(lib().bitnet_i8_linear_workspace_bytes(M, K))


def bitnet_i8_linear_into(M, N, K, x, q, w_scale, bias, relu, y, workspace, acc_out=None,
                          stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().bitnet_i8_linear(M, N, K, _ptr(x), _ptr(q), _ptr(w_scale), _ptr(bias),
                                  int(bool(relu)), _ptr(y), _ptr(workspace), ws_bytes,
                                  _ptr(acc_out), _stream(stream)),
           "bitnet_i8_linear")


def bitnet_i8_linear(x: torch.Tensor, q: torch.Tensor, w_scale: torch.Tensor, bias=None,
                     relu: bool = False, return_acc: bool = False, stream=None):
    """I8_S layer: fp32 x [M,K], int8 q [N,K] -> fp32 y [M,N] (and int32 acc)."""
    _dev(x, torch.float32, "x")
    _dev(q, torch.int8, "q")
    M, K = x.shape
    N = q.shape[0]
    y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    ws = torch.empty(bitnet_i8_linear_workspace_bytes(M, K), dtype=torch.uint8, device=x.device)
    acc = torch.empty((M, N), dtype=torch.int32, device=x.device) if return_acc else None
    bitnet_i8_linear_into(M, N, K, x, q, w_scale, bias, relu, y, ws, acc, stream)
    return (y, acc) if return_acc else y


# ---- the 8-bit table with one scale per row: embeddings and lm_head ---------

def bitnet_i8_quant_weights_rows_into(W, N, K, q, w_scale, stream=None) -> None:
    _check(lib().bitnet_i8_quant_weights_rows(_ptr(W), N, K, _ptr(q), _ptr(w_scale),
                                              _stream(stream)),
           "bitnet_i8_quant_weights_rows")


def bitnet_i8_quant_weights_rows(W: torch.Tensor, stream=None):
    """fp32 W [N,K] -> (q int8 [N,K], w_scale fp32 [N]): one absmax scale per row."""
    _dev(W, torch.float32, "W")
    N, K = W.shape
    q = torch.empty((N, K), dtype=torch.int8, device=W.device)
    w_scale = torch.empty(N, dtype=torch.float32, device=W.device)
    bitnet_i8_quant_weights_rows_into(W, N, K, q, w_scale, stream)
    return q, w_scale


def bitnet_table_bytes(V: int, K: int) -> int:
    return int(lib().bitnet_table_bytes(V, K))


def bitnet_table_quant_into(W, V, K, table, w_scale, stream=None) -> None:
    _check(lib().bitnet_table_quant(_ptr(W), V, K, _ptr(table), _ptr(w_scale), _stream(stream)),
           "bitnet_table_quant")


def bitnet_table_quant(W: torch.Tensor, stream=None):
    """fp32 W [V,K] -> (table int8 [bitnet_table_bytes(V, K)] in the library's
    storage order, w_scale fp32 [V])."""
    _dev(W, torch.float32, "W")
    V, K = W.shape
    table = torch.empty(bitnet_table_bytes(V, K), dtype=torch.int8, device=W.device)
    w_scale = torch.empty(V, dtype=torch.float32, device=W.device)
    bitnet_table_quant_into(W, V, K, table, w_scale, stream)
    return table, w_scale


def bitnet_embed_lookup_into(ids, T, table, w_scale, V, K, out, stream=None) -> None:
    _check(lib().bitnet_embed_lookup(_ptr(ids), T, _ptr(table), _ptr(w_scale), V, K, _ptr(out),
                                     _stream(stream)),
           "bitnet_embed_lookup")


def bitnet_embed_lookup(ids: torch.Tensor, table: torch.Tensor, w_scale: torch.Tensor, K: int,
                        stream=None):
    """int32 token ids [T] -> fp32 embedding rows [T, K] of the table (V = w_scale.numel())."""
    _dev(ids, torch.int32, "ids")
    _dev(table, torch.int8, "table")
    V = w_scale.numel()
    T = ids.numel()
    out = torch.empty((T, K), dtype=torch.float32, device=table.device)
    bitnet_embed_lookup_into(ids, T, table, w_scale, V, K, out, stream)
    return out


def bitnet_lm_head_into(M, V, K, x, table, w_scale, y, xq_out=None, x_scale_out=None,
                        acc_out=None, stream=None) -> None:
    _check(lib().bitnet_lm_head(M, V, K, _ptr(x), _ptr(table), _ptr(w_scale), _ptr(y),
                                _ptr(xq_out), _ptr(x_scale_out), _ptr(acc_out), _stream(stream)),
           "bitnet_lm_head")


def bitnet_lm_head(x: torch.Tensor, table: torch.Tensor, w_scale: torch.Tensor,
                   return_parts: bool = False, stream=None):
    """lm_head over the table: fp32 x [M,K] (M <= 16) -> fp32 logits [M, V]
    (V = w_scale.numel()); with return_parts, a dict that also holds xq,
    x_scale and the int32 acc."""
    _dev(x, torch.float32, "x")
    _dev(table, torch.int8, "table")
    M, K = x.shape
    V = w_scale.numel()
    y = torch.empty((M, V), dtype=torch.float32, device=x.device)
    if not return_parts:
        bitnet_lm_head_into(M, V, K, x, table, w_scale, y, stream=stream)
        return y
    xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    xs = torch.empty(M, dtype=torch.float32, device=x.device)
    acc = torch.empty((M, V), dtype=torch.int32, device=x.device)
    bitnet_lm_head_into(M, V, K, x, table, w_scale, y, xq, xs, acc, stream)
    return {"y": y, "xq": xq, "x_scale": xs, "acc": acc}


def bitnet_i8_linear_rows_into(M, N, K, x, q, w_scale, bias, relu, y, workspace, acc_out=None,
                               stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().bitnet_i8_linear_rows(M, N, K, _ptr(x), _ptr(q), _ptr(w_scale), _ptr(bias),
                                       int(bool(relu)), _ptr(y), _ptr(workspace), ws_bytes,
                                       _ptr(acc_out), _stream(stream)),
           "bitnet_i8_linear_rows")


def bitnet_i8_linear_rows(x: torch.Tensor, q: torch.Tensor, w_scale: torch.Tensor, bias=None,
                          relu: bool = False, return_acc: bool = False, stream=None):
    """I8_S layer with per-channel weight scales: fp32 x [M,K], int8 q [N,K],
    fp32 w_scale [N] -> fp32 y [M,N] (and int32 acc)."""
    _dev(x, torch.float32, "x")
    _dev(q, torch.int8, "q")
    M, K = x.shape
    N = q.shape[0]
    y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    ws = torch.empty(bitnet_i8_linear_workspace_bytes(M, K), dtype=torch.uint8, device=x.device)
    acc = torch.empty((M, N), dtype=torch.int32, device=x.device) if return_acc else None
    bitnet_i8_linear_rows_into(M, N, K, x, q, w_scale, bias, relu, y, ws, acc, stream)
    return (y, acc) if return_acc else y


# ---- I8_S causal depthwise convolution ---------------------------------------

def bitnet_i8_dwconv_quant_weights(W: torch.Tensor, stream=None):
    """fp32 kernel W [C,k] -> (q int8 [C,k], w_scale fp32 [C]), per channel."""
    _dev(W, torch.float32, "W")
    C, k = W.shape
    q = torch.empty((C, k), dtype=torch.int8, device=W.device)
    s = torch.empty(C, dtype=torch.float32, device=W.device)
    _check(lib().bitnet_i8_dwconv_quant_weights(_ptr(W), C, k, _ptr(q), _ptr(s), _stream(stream)),
           "bitnet_i8_dwconv_quant_weights")
    return q, s


def bitnet_i8_dwconv_workspace_bytes(B: int, T: int, C: int) -> int:
    return int(lib().bitnet_i8_dwconv_workspace_bytes(B, T, C))


def bitnet_i8_dwconv_into(B, T, C, k, x, q, w_scale, bias, relu, y, workspace, acc_out=None,
                          x_scale_out=None, stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().bitnet_i8_dwconv(B, T, C, k, _ptr(x), _ptr(q), _ptr(w_scale), _ptr(bias),
                                  int(bool(relu)), _ptr(y), _ptr(workspace), ws_bytes,
                                  _ptr(acc_out), _ptr(x_scale_out), _stream(stream)),
           "bitnet_i8_dwconv")


def bitnet_i8_dwconv(x: torch.Tensor, q: torch.Tensor, w_scale: torch.Tensor, bias=None,
                     relu: bool = False, return_parts: bool = False, stream=None):
    """Causal depthwise convolution over frames: fp32 x [B,T,C], int8 q [C,k] ->
    fp32 y [B,T,C] (with return_parts, a dict that also holds acc and x_scale)."""
    _dev(x, torch.float32, "x")
    _dev(q, torch.int8, "q")
    B, T, C = x.shape
    k = q.shape[1]
    y = torch.empty((B, T, C), dtype=torch.float32, device=x.device)
    ws = torch.empty(bitnet_i8_dwconv_workspace_bytes(B, T, C), dtype=torch.uint8,
                     device=x.device)
    if not return_parts:
        bitnet_i8_dwconv_into(B, T, C, k, x, q, w_scale, bias, relu, y, ws, stream=stream)
        return y
    acc = torch.empty((B, T, C), dtype=torch.int32, device=x.device)
    xs = torch.empty((B, C), dtype=torch.float32, device=x.device)
    bitnet_i8_dwconv_into(B, T, C, k, x, q, w_scale, bias, relu, y, ws, acc, xs, stream)
    return {"y": y, "acc": acc, "x_scale": xs}


def bitnet_ternary_matmul_lut_grouped(problems_dev, count, problems_host, stream=None) -> None:
    _check(lib().bitnet_ternary_matmul_lut_grouped(_ptr(problems_dev), count,
                                                   _c.byref(problems_host), _stream(stream)),
           "bitnet_ternary_matmul_lut_grouped")


class LutPlan:
    """Independent single-row projections run by the lookup-table kernel in one
    launch (the comparison variant of the grouped decode call at M = 1)."""

    def __init__(self, xs, packeds, w_scales, ys, Ns, Ks, device=None):
        count = len(xs)
        if not 1 <= count <= BITNET_MAX_GROUP:
            raise ValueError(f"group size must be 1..{BITNET_MAX_GROUP}")
        arr = (bitnet_problem * count)()
        for i in range(count):
            arr[i] = bitnet_problem(xs[i].data_ptr(), packeds[i].data_ptr(),
                                    w_scales[i].data_ptr(), ys[i].data_ptr(), int(Ns[i]),
                                    int(Ks[i]))
        self._keep = (list(xs), list(packeds), list(w_scales), list(ys))
        self.host, self.count = arr, count
        dev = device if device is not None else xs[0].device
        self.dev = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8).to(dev)

    def run(self, stream=None) -> None:
        bitnet_ternary_matmul_lut_grouped(self.dev, self.count, self.host, stream)


def bitnet_stages_workspace_bytes(M: int, problems_host, count: int) -> int:
    return int(lib().bitnet_stages_workspace_bytes(M, _c.byref(problems_host), count))


def bitnet_ternary_matmul_stages(M, problems_dev, count, stage_end_host, nstages, problems_host,
                                 workspace, stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().bitnet_ternary_matmul_stages(M, _ptr(problems_dev), count,
                                              _c.byref(stage_end_host), nstages,
                                              _c.byref(problems_host), _ptr(workspace), ws_bytes,
                                              _stream(stream)),
           "bitnet_ternary_matmul_stages")


class StagedPlan:
    """A fixed sequence of dependent stages of decode projections (for example
    one token through a decoder: q,k,v | o | gate,up | down per layer), run by
    one call.  stages: list of lists of (x, packed, w_scale, y, N, K) tuples; a
    problem whose x is the y tensor of a problem of an earlier stage reads that
    output.  The workspace is zero-filled here, once."""

    def __init__(self, M: int, stages, device=None):
        flat = [pr for st in stages for pr in st]
        count = len(flat)
        if not 1 <= count <= BITNET_MAX_GROUP:
            raise ValueError(f"at most {BITNET_MAX_GROUP} problems")
        self.M, self.count, self.nstages = int(M), count, len(stages)
        arr = (bitnet_problem * count)()
        for i, (x, pk, ws, y, N, K) in enumerate(flat):
            arr[i] = bitnet_problem(x.data_ptr(), pk.data_ptr(), ws.data_ptr(), y.data_ptr(),
                                    int(N), int(K))
        ends = (_i32 * self.nstages)()
        e = 0
        for s, st in enumerate(stages):
            e += len(st)
            ends[s] = e
        self._keep = flat
        self.host, self.ends = arr, ends
        dev = device if device is not None else flat[0][0].device
        self.dev = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8).to(dev)
        nbytes = bitnet_stages_workspace_bytes(self.M, arr, count)
        if nbytes == 0:
            raise ValueError("invalid staged problem list")
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=dev)

    def run(self, stream=None) -> None:
        bitnet_ternary_matmul_stages(self.M, self.dev, self.count, self.ends, self.nstages,
                                     self.host, self.workspace, stream)

    def timed_out(self) -> bool:
        """After the call has completed: did a wait between stages run out?"""
        return int(self.workspace[4:8].view(torch.int32).item()) != 0

    def timeouts_total(self) -> int:
        """Calls with a wait that ran out, since the workspace was zero-filled."""
        return int(self.workspace[8:12].view(torch.int32).item())


# ---- the paged key-value cache and beam search ------------------------------

KV_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.int8: 2}


class KvCache:
    """The keys and values of all layers in pages.

    k, v: device tensors [layers, pages, kv_heads, page_size, head_dim] of
    bfloat16, float16 or int8, with equal strides and contiguous channels (heads
    before tokens in memory, or a transposed view of tokens before heads).
    int8 caches carry fp32 scales k_scale, v_scale [layers, pages, kv_heads,
    page_size].  Holds the descriptor that the calls pass to the library.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale=None, v_scale=None):
        if k.dtype not in KV_DTYPES:
            raise ValueError(f"cache dtype must be one of {list(KV_DTYPES)}, got {k.dtype}")
        if k.dim() != 5 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be [layers, pages, kv_heads, page_size, head_dim] alike")
        layers, pages, heads, page, dim = k.shape
        if not (k.is_cuda and v.device == k.device):
            raise ValueError("k and v must be device tensors of one device")
        # strides of axes of one entry are never used and may be anything
        if any(n > 1 and a != b for n, a, b in zip(k.shape, k.stride(), v.stride())):
            raise ValueError("k and v must have equal strides")
        if dim > 1 and k.stride(4) != 1:
            raise ValueError("channels must be contiguous")
        if (k.dtype is torch.int8) != (k_scale is not None and v_scale is not None) or (
                (k_scale is None) != (v_scale is None)):
            raise ValueError("int8 caches, and no others, take k_scale and v_scale")
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is not None:
                _dev(t, torch.float32, name)
                if t.shape != k.shape[:4] or t.device != k.device:
                    raise ValueError(f"{name} must be [layers, pages, kv_heads, page_size]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.layers, self.pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        st = [s if n > 1 else max(dim, 16) for n, s in zip(k.shape, k.stride())]
        self.c = bitnet_kv_cache(
            k.data_ptr(), v.data_ptr(), 0 if k_scale is None else k_scale.data_ptr(),
            0 if v_scale is None else v_scale.data_ptr(), st[0], st[1], st[2], st[3],
            KV_DTYPES[k.dtype], layers, pages, heads, page, dim)
        self.ref = _c.byref(self.c)

    @classmethod
    def empty(cls, layers: int, pages: int, kv_heads: int, page_size: int, head_dim: int,
              dtype=torch.bfloat16, device="cuda"):
        """A cache of uninitialized pages, heads before tokens."""
        shape = (layers, pages, kv_heads, page_size, head_dim)
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        if dtype is not torch.int8:
            return cls(k, v)
        return cls(k, v, *(torch.empty(shape[:4], dtype=torch.float32, device=device)
                           for _ in range(2)))


class KvPool:
    """The pages of a set of requests: block tables, the pages each request
    owns and the stack of unused pages (int32 device tensors)."""

    def __init__(self, pages: int, page_size: int, tables: torch.Tensor, owned: torch.Tensor,
                 free_pages: torch.Tensor):
        for t, name in ((tables, "tables"), (owned, "owned"), (free_pages, "free_pages")):
            _dev(t, torch.int32, name)
            if t.device != tables.device:
                raise ValueError(f"{name} is on another device than tables")
        if tables.dim() != 2 or owned.shape != tables.shape or free_pages.numel() != pages:
            raise ValueError("tables and owned are [rows, max_pages], free_pages [pages]")
        self.tables, self.owned, self.free_pages = tables, owned, free_pages
        self.rows, self.max_pages = tables.shape
        self.pages, self.page_size = int(pages), int(page_size)
        self.c = bitnet_kv_pool(tables.data_ptr(), owned.data_ptr(), free_pages.data_ptr(),
                                self.rows, self.max_pages, self.pages, self.page_size)
        self.ref = _c.byref(self.c)

    @classmethod
    def empty(cls, rows: int, max_pages: int, pages: int, page_size: int, device="cuda"):
        """(pool, state) of requests without tokens; all pages are free, and
        the lowest numbered ones are handed out first."""
        i32 = dict(dtype=torch.int32, device=device)
        tables, owned = (torch.full((rows, max_pages), -1, **i32) for _ in range(2))
        free = torch.arange(pages - 1, -1, -1, **i32)
        state = torch.zeros(2 * rows + 1, **i32)
        state[-1] = pages
        return cls(pages, page_size, tables, owned, free), state


def bitnet_kv_map_into(pool: KvPool, T, new_lens, state_in, state_out, starts, slots, positions,
                       rows, status, stream=None) -> None:
    _check(lib().bitnet_kv_map(pool.ref, T, _ptr(new_lens), _ptr(state_in), _ptr(state_out),
                               _ptr(starts), _ptr(slots), _ptr(positions), _ptr(rows),
                               _ptr(status), _stream(stream)),
           "bitnet_kv_map")


def _rows_stride(t, width):
    """Elements between the rows of a [T, width] tensor with contiguous rows."""
    return t.stride(0) if t.size(0) > 1 else max(width, 4)


def bitnet_kv_append_into(cache: KvCache, layer, T, q_heads, k, v, slots, positions=None, cos=None,
                          sin=None, q=None, q_out=None, stream=None) -> None:
    w = cache.kv_heads * cache.head_dim
    _check(lib().bitnet_kv_append(cache.ref, layer, T, q_heads, _ptr(k), _rows_stride(k, w),
                                  _ptr(v), _rows_stride(v, w), _ptr(slots), _ptr(positions),
                                  _ptr(cos), _ptr(sin), 0 if cos is None else cos.size(0),
                                  _ptr(q),
                                  0 if q is None else _rows_stride(q, q_heads * cache.head_dim),
                                  _ptr(q_out), _stream(stream)),
           "bitnet_kv_append")


def bitnet_paged_attention_workspace_bytes(T: int, q_heads: int, kv_heads: int, head_dim: int,
                                           max_len: int) -> int:
    return int(lib().bitnet_paged_attention_workspace_bytes(T, q_heads, kv_heads, head_dim,
                                                            max_len))


def bitnet_paged_attention_into(cache: KvCache, layer, T, q_heads, q, tables, lens, max_len, scale,
                                out, workspace, rows=None, lse=None, stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().bitnet_paged_attention(cache.ref, layer, T, q_heads, _ptr(q),
                                        _rows_stride(q, q_heads * cache.head_dim), _ptr(tables),
                                        tables.size(0), tables.size(1), _ptr(rows), _ptr(lens),
                                        max_len, scale, _ptr(out), _ptr(lse), _ptr(workspace),
                                        ws_bytes, _stream(stream)),
           "bitnet_paged_attention")


def bitnet_beam_select_workspace_bytes(B: int, W: int, V: int) -> int:
    return int(lib().bitnet_beam_select_workspace_bytes(B, W, V))


def bitnet_beam_select_into(B, W, V, logits, scores_in, finished_in, eos, scores_out, tokens,
                            parents, finished_out, workspace, stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().bitnet_beam_select(B, W, V, _ptr(logits), _rows_stride(logits, V),
                                    _ptr(scores_in), _ptr(finished_in), eos, _ptr(scores_out),
                                    _ptr(tokens), _ptr(parents), _ptr(finished_out),
                                    _ptr(workspace), ws_bytes, _stream(stream)),
           "bitnet_beam_select")


def bitnet_beam_reorder_into(cache: KvCache, B, W, parents, lens, tables_in, tables_out,
                             stream=None) -> None:
    _check(lib().bitnet_beam_reorder(cache.ref, B, W, _ptr(parents), _ptr(lens), _ptr(tables_in),
                                     _ptr(tables_out), tables_in.size(1), _stream(stream)),
           "bitnet_beam_reorder")


# Convenience forms: arguments checked against the cache's and the pool's
# shapes, outputs (and workspaces) allocated with torch on the stream that runs
# the call.

def _on(stream):
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _here(dev: torch.device, stream=None) -> None:
    if dev.index is not None and dev.index != torch.cuda.current_device():
        raise ValueError(f"tensors of {dev}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if stream is not None and stream.device != dev:
        raise ValueError(f"a stream of {stream.device}, but tensors of {dev}")


def _arg(t: torch.Tensor, dtype, shape, dev: torch.device, name: str) -> None:
    _dev(t, dtype, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not on {dev}")


def _rows_arg(t: torch.Tensor, T: int, width: int, dev: torch.device, name: str) -> None:
    """fp32 [T, width] whose rows are contiguous and may lie apart."""
    if not t.is_cuda or t.dtype != torch.float32 or t.device != dev:
        raise ValueError(f"{name} must be a torch.float32 tensor on {dev}")
    if t.dim() != 2 or tuple(t.shape) != (T, width) or (width > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [{T}, {width}] with contiguous rows")


def bitnet_kv_map(pool: KvPool, T: int, new_lens: torch.Tensor, state: torch.Tensor, stream=None):
    """One step's tokens: new_lens int32 [rows] (tokens to add, 0, or negative to
    end a request) and state int32 [2*rows + 1], which is updated in place ->
    dict of starts [rows + 1], slots, positions, rows [T] and status [rows]."""
    dev = pool.tables.device
    _here(dev, stream)
    _arg(new_lens, torch.int32, (pool.rows,), dev, "new_lens")
    _arg(state, torch.int32, (2 * pool.rows + 1,), dev, "state")
    with _on(stream):
        out = {n: torch.empty(c, dtype=torch.int32, device=dev)
               for n, c in (("starts", pool.rows + 1), ("slots", T), ("positions", T), ("rows", T),
                            ("status", pool.rows))}
        bitnet_kv_map_into(pool, T, new_lens, state, state, *out.values(), stream=stream)
    return out


def bitnet_kv_append(cache: KvCache, layer: int, k: torch.Tensor, v: torch.Tensor,
                     slots: torch.Tensor, positions=None, cos=None, sin=None, q=None, stream=None):
    """Write fp32 rows k, v [T, kv_heads*head_dim] to the slots of one layer; with
    cos and sin [max_pos, head_dim/2] k and q [T, q_heads*head_dim] are rotated
    by their positions first.  Returns the rotated q (None without q)."""
    dev, D = cache.k.device, cache.head_dim
    _here(dev, stream)
    T = k.shape[0]
    _rows_arg(k, T, cache.kv_heads * D, dev, "k")
    _rows_arg(v, T, cache.kv_heads * D, dev, "v")
    _arg(slots, torch.int32, (T,), dev, "slots")
    if (cos is None) != (sin is None) or (cos is not None and positions is None):
        raise ValueError("a rotation takes cos, sin and positions")
    if cos is not None:
        _arg(cos, torch.float32, (cos.shape[0], D // 2), dev, "cos")
        _arg(sin, torch.float32, cos.shape, dev, "sin")
        _arg(positions, torch.int32, (T,), dev, "positions")
    q_heads, q_out = 0, None
    with _on(stream):
        if q is not None:
            q_heads = q.shape[1] // D
            _rows_arg(q, T, q_heads * D, dev, "q")
            q_out = torch.zeros((T, q_heads * D), dtype=torch.float32, device=dev)
        bitnet_kv_append_into(cache, layer, T, q_heads, k, v, slots, positions, cos, sin, q, q_out,
                              stream)
    return q_out


def bitnet_paged_attention(cache: KvCache, layer: int, q: torch.Tensor, tables: torch.Tensor,
                           lens: torch.Tensor, max_len=None, scale=None, rows=None,
                           return_lse: bool = False, stream=None):
    """Attention of q fp32 [T, q_heads*head_dim], one new token per row, over the
    first lens[t] tokens of table row rows[t] (default t).  max_len defaults to
    what a table holds, scale to head_dim**-0.5.  Returns fp32 [T,
    q_heads*head_dim] (and the log-sum-exp [T, q_heads])."""
    dev, D = cache.k.device, cache.head_dim
    _here(dev, stream)
    T, width = q.shape
    _rows_arg(q, T, width, dev, "q")
    if width % (cache.kv_heads * D):
        raise ValueError("q's width must be a multiple of kv_heads*head_dim")
    if tables.dim() != 2:
        raise ValueError("tables must be [rows, max_pages]")
    _arg(tables, torch.int32, tables.shape, dev, "tables")
    _arg(lens, torch.int32, (T,), dev, "lens")
    if rows is not None:
        _arg(rows, torch.int32, (T,), dev, "rows")
    if max_len is None:
        max_len = tables.shape[1] * cache.page_size
    H = width // D
    with _on(stream):
        out = torch.empty((T, width), dtype=torch.float32, device=dev)
        lse = torch.empty((T, H), dtype=torch.float32, device=dev) if return_lse else None
        ws = torch.zeros(bitnet_paged_attention_workspace_bytes(T, H, cache.kv_heads, D, max_len),
                         dtype=torch.uint8, device=dev)
        bitnet_paged_attention_into(cache, layer, T, H, q, tables, lens, max_len,
                                    D ** -0.5 if scale is None else scale, out, ws, rows, lse,
                                    stream)
    return (out, lse) if return_lse else out


def bitnet_beam_select(logits: torch.Tensor, scores: torch.Tensor, W: int, finished=None,
                       eos: int = -1, stream=None):
    """The next W beams of each group: fp32 logits [B*W, V] (rows may lie apart),
    scores [B*W], optional finished flags int32 [B*W] with the end token eos ->
    dict of scores, tokens, parents (row numbers) and, with finished, finished."""
    dev = logits.device
    _here(dev, stream)
    R, V = logits.shape
    _rows_arg(logits, R, V, dev, "logits")
    if W < 1 or R % W:
        raise ValueError("logits rows must be a multiple of W")
    _arg(scores, torch.float32, (R,), dev, "scores")
    if finished is not None:
        _arg(finished, torch.int32, (R,), dev, "finished")
    with _on(stream):
        out = {"scores": torch.empty(R, dtype=torch.float32, device=dev)}
        for n in ("tokens", "parents") + (("finished",) if finished is not None else ()):
            out[n] = torch.empty(R, dtype=torch.int32, device=dev)
        ws = torch.zeros(bitnet_beam_select_workspace_bytes(R // W, W, V), dtype=torch.uint8,
                         device=dev)
        bitnet_beam_select_into(R // W, W, V, logits, scores, finished, eos, out["scores"],
                                out["tokens"], out["parents"], out.get("finished"), ws, stream)
    return out


def bitnet_beam_reorder(cache: KvCache, tables: torch.Tensor, lens: torch.Tensor,
                        parents: torch.Tensor, W: int, stream=None):
    """The block tables [B*W, max_pages] of the beams that continue parents
    (row numbers); partly filled last pages are copied inside the cache.
    Returns new tables; the old ones are unchanged."""
    dev = cache.k.device
    _here(dev, stream)
    if tables.dim() != 2 or W < 1 or tables.shape[0] % W:
        raise ValueError("tables must be [B*W, max_pages]")
    R = tables.shape[0]
    _arg(tables, torch.int32, tables.shape, dev, "tables")
    _arg(lens, torch.int32, (R,), dev, "lens")
    _arg(parents, torch.int32, (R,), dev, "parents")
    with _on(stream):
        out = torch.empty_like(tables)
        bitnet_beam_reorder_into(cache, R // W, W, parents, lens, tables, out, stream)
    return out
