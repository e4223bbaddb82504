"""MI355X-native W4A16 group-wise quantized linear layer (AWQ's WQLinear hot path).

A thin binding of the C ABI in ``include/awq.h`` (``libawq_mi355x.so``, built
by ``python -m bit_weight_only_awq_amd.build``).  PyTorch supplies device
memory and the current stream only; every step of the layer runs in the
library's HIP kernels.  There is no fallback: if the library is missing or
the tensors are not on the GPU, the calls raise.

Entry points (same names and arguments as the C ABI):

* ``awq_pack(w, group_size, zero_point)`` -> ``(qweight, scales, qzeros)``
* ``awq_dequant(qweight, scales, qzeros, N, K, group_size, zero_point)``
* ``awq_gemv(x, qweight, scales, qzeros, N, K, group_size, zero_point)``
* ``awq_gemm(x, qweight, scales, qzeros, N, K, group_size, zero_point)``
* ``awq_gemm_workspace_bytes(M, N, K, group_size)``, ``awq_strerror(status)``

plus ``pack(W, q_group_size, zero_point)`` / ``linear(x, packed)`` which pick
GEMV up to 8 tokens and GEMM otherwise, following ``quant_config``'s
``version`` ("Optimization Awq", section "Quantizar seu próprio modelo").

The layer with its epilogue and the layers of experts:

* ``linear_fused(x, packed, bias, activation, gated, residual)``
* ``route_experts(logits, top_k, renormalize)`` -> ``ExpertRoute``
* ``pack_experts(W, q_group_size, zero_point)`` -> ``PackedExperts``
* ``linear_experts(x, experts, route, bias, activation, gated)``
* ``combine_experts(h, experts, route, bias, residual)``
* ``expert_mlp(x, logits, gate_up, down, top_k)``: the four together

``mlp(x, gate_up, down, residual)``, a decoder block's MLP in two launches, and
the block's other half on a paged cache of keys and values:

* ``kv_cache(pages, kv_heads, head_dim, page_size)`` -> ``KvCache``, ``Sequences(offsets, lengths, tables)``
* ``append_kv(qkv, cache, seqs, inv_freq)`` -> rotated queries
* ``attend(q, cache, seqs, scale, shared)``
* ``select_pages(q, cache, seqs, count)``, ``attend_pages(q, cache, seqs, pages)``
* ``attention(x, qkv, o, cache, seqs, inv_freq)``: the layers and the calls above together
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple, Optional

import torch  # noqa: F401  (loaded first: the library then shares torch's HIP runtime)

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libawq_mi355x.so")

AWQ_OK = 0
AWQ_ERR_NULL = -1
AWQ_ERR_SHAPE = -2
AWQ_ERR_GROUP = -3
AWQ_ERR_ALIGN = -4
AWQ_ERR_UNSUPPORTED = -5
AWQ_ERR_WORKSPACE = -6
AWQ_ERR_HIP = -7
AWQ_ERR_SCRATCH = -8
AWQ_ERR_OPTION = -9

# awq_activation: the activations of the fused layers' epilogue
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

EXPORTED = ("awq_pack", "awq_dequant", "awq_gemv", "awq_gemm", "awq_gemm_workspace_bytes", "awq_strerror",
            "awq_scale_candidates", "awq_scale_candidates_workspace_bytes", "awq_scale_loss",
            "awq_scale_loss_workspace_bytes", "awq_scale_columns", "awq_clip_search",
            "awq_clip_search_workspace_bytes", "awq_scale_search", "awq_scale_search_workspace_bytes",
            "awq_gemm_noalloc", "awq_gemm_noalloc_max_workspace_bytes",
            "awq_linear_fused", "awq_linear_fused_workspace_bytes", "awq_route_experts",
            "awq_route_experts_workspace_bytes", "awq_linear_experts", "awq_linear_experts_workspace_bytes",
            "awq_combine_experts", "awq_combine_experts_workspace_bytes",
            "awq_append_kv", "awq_attend", "awq_attend_workspace_bytes", "awq_select_pages",
            "awq_select_pages_workspace_bytes", "awq_attend_pages", "awq_attend_pages_workspace_bytes")

_lib: Optional[ctypes.CDLL] = None


class AwqError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {awq_strerror(status)} (status {status})")
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the C ABI library once; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m bit_weight_only_awq_amd.build` (hipcc, gfx950)")
    lib = ctypes.CDLL(path)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.awq_pack.argtypes = [P, I32, I32, I32, I32, P, P, P, P]
    lib.awq_pack.restype = ctypes.c_int
    lib.awq_dequant.argtypes = [P, P, P, P, I32, I32, I32, I32, P]
    lib.awq_dequant.restype = ctypes.c_int
    lib.awq_gemv.argtypes = [P, P, P, P, P, I32, I32, I32, I32, I32, P]
    lib.awq_gemv.restype = ctypes.c_int
    lib.awq_gemm.argtypes = [P, P, P, P, P, I32, I32, I32, I32, I32, P, SZ, P]
    lib.awq_gemm.restype = ctypes.c_int
    lib.awq_gemm_workspace_bytes.argtypes = [I32, I32, I32, I32]
    lib.awq_gemm_workspace_bytes.restype = SZ
    lib.awq_strerror.argtypes = [ctypes.c_int]
    lib.awq_strerror.restype = ctypes.c_char_p
    lib.awq_scale_candidates.argtypes = [P, I32, I32, P, I32, I32, P, I32, P, P, SZ, P]
    lib.awq_scale_candidates.restype = ctypes.c_int
    lib.awq_scale_candidates_workspace_bytes.argtypes = [I32, I32, I32]
    lib.awq_scale_candidates_workspace_bytes.restype = SZ
    lib.awq_scale_search.argtypes = [P, P, I32, I32, I32, I32, I32, P, I32, I32, P, P, P, P, SZ, P]
    lib.awq_scale_search.restype = ctypes.c_int
    lib.awq_scale_search_workspace_bytes.argtypes = [I32, I32, I32, I32]
    lib.awq_scale_search_workspace_bytes.restype = SZ
    lib.awq_gemm_noalloc.argtypes = [P, P, P, P, P, I32, I32, I32, I32, I32, P]
    lib.awq_gemm_noalloc.restype = ctypes.c_int
    lib.awq_gemm_noalloc_max_workspace_bytes.argtypes = []
    lib.awq_gemm_noalloc_max_workspace_bytes.restype = SZ
    lib.awq_scale_loss.argtypes = [P, P, P, I32, I32, I32, I32, I32, I32, P, SZ, P, P]
    lib.awq_scale_loss.restype = ctypes.c_int
    lib.awq_scale_loss_workspace_bytes.argtypes = [I32, I32, I32, I32]
    lib.awq_scale_loss_workspace_bytes.restype = SZ
    lib.awq_scale_columns.argtypes = [P, I32, I32, P, I32, P, P]
    lib.awq_scale_columns.restype = ctypes.c_int
    lib.awq_clip_search.argtypes = [P, P, I32, I32, I32, I32, I32, P, I32, P, P, P, SZ, P]
    lib.awq_clip_search.restype = ctypes.c_int
    lib.awq_clip_search_workspace_bytes.argtypes = [I32, I32, I32, I32, I32]
    lib.awq_clip_search_workspace_bytes.restype = SZ
    lib.awq_linear_fused.argtypes = [P, I32, P, P, P, P, I32, I32, P, I32, P, I32, I32, I32, I32, I32, I32, P, SZ, P]
    lib.awq_linear_fused.restype = ctypes.c_int
    lib.awq_linear_fused_workspace_bytes.argtypes = [I32, I32, I32, I32, I32]
    lib.awq_linear_fused_workspace_bytes.restype = SZ
    lib.awq_route_experts.argtypes = [P, I32, I32, I32, I32, I32, I32, P, P, P, P, P, P, SZ, P]
    lib.awq_route_experts.restype = ctypes.c_int
    lib.awq_route_experts_workspace_bytes.argtypes = [I32, I32]
    lib.awq_route_experts_workspace_bytes.restype = SZ
    lib.awq_linear_experts.argtypes = [P, I32, I32, P, I32, P, I32, I32, P, P, P, P, I32, I32, P, I32, I32, I32, I32,
                                       I32, P, SZ, P]
    lib.awq_linear_experts.restype = ctypes.c_int
    lib.awq_linear_experts_workspace_bytes.argtypes = [I32, I32, I32, I32, I32, I32]
    lib.awq_linear_experts_workspace_bytes.restype = SZ
    lib.awq_combine_experts.argtypes = [P, I32, P, P, P, I32, I32, I32, P, P, P, P, P, I32, P, I32, I32, I32, I32, I32,
                                        P, SZ, P]
    lib.awq_combine_experts.restype = ctypes.c_int
    lib.awq_combine_experts_workspace_bytes.argtypes = [I32, I32, I32, I32, I32, I32]
    lib.awq_combine_experts_workspace_bytes.restype = SZ
    F32 = ctypes.c_float
    batch = [P, P, P, I32, I32, I32, I32, I32, I32]  # offsets, lengths, tables, width, T, B, q_heads, kv_heads, head_dim
    lib.awq_append_kv.argtypes = [P, I32, *batch, P, I32, I32, P, I32, P, P, I32, P, P, P, I32, I32, P]
    lib.awq_append_kv.restype = ctypes.c_int
    lib.awq_attend.argtypes = [P, I32, *batch, F32, I32, P, P, I32, I32, P, I32, P, SZ, P]
    lib.awq_attend.restype = ctypes.c_int
    lib.awq_attend_workspace_bytes.argtypes = [I32] * 8
    lib.awq_attend_workspace_bytes.restype = SZ
    lib.awq_select_pages.argtypes = [P, I32, *batch, P, I32, I32, I32, I32, I32, P, P, SZ, P]
    lib.awq_select_pages.restype = ctypes.c_int
    lib.awq_select_pages_workspace_bytes.argtypes = [I32] * 4
    lib.awq_select_pages_workspace_bytes.restype = SZ
    lib.awq_attend_pages.argtypes = [P, I32, *batch, F32, P, I32, P, P, I32, I32, P, I32, P, SZ, P]
    lib.awq_attend_pages.restype = ctypes.c_int
    lib.awq_attend_pages_workspace_bytes.argtypes = [I32] * 6
    lib.awq_attend_pages_workspace_bytes.restype = SZ
    _lib = lib
    return lib


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the AWQ kernels must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the AWQ kernels must be contiguous")
    return t.data_ptr()


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _check(status: int, where: str) -> None:
    if status != AWQ_OK:
        raise AwqError(status, where)


def awq_strerror(status: int) -> str:
    return load_library().awq_strerror(int(status)).decode()


def awq_gemm_workspace_bytes(M: int, N: int, K: int, group_size: int) -> int:
    return int(load_library().awq_gemm_workspace_bytes(M, N, K, group_size))


def awq_pack(w: torch.Tensor, group_size: int = 128, zero_point: bool = True,
             qweight: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
             qzeros: Optional[torch.Tensor] = None):
    """Quantize fp16 ``w`` [N, K] and return ``(qweight int32 [N, K/8], scales fp16 [N/8, K/g, 8],
    qzeros int32 [N/8, K/g] or None)``; the int32 tensors hold the ABI's uint32 words."""
    lib = load_library()
    if w.dtype != torch.float16 or w.dim() != 2:
        raise ValueError("w must be a 2-D float16 tensor [N, K]")
    N, K = w.shape
    G = K // group_size if group_size > 0 else 0
    dev = w.device
    if qweight is None:
        qweight = torch.empty((N, K // 8), dtype=torch.int32, device=dev)
    if scales is None:
        scales = torch.empty((N // 8, G, 8), dtype=torch.float16, device=dev)
    if zero_point and qzeros is None:
        qzeros = torch.empty((N // 8, G), dtype=torch.int32, device=dev)
    st = lib.awq_pack(_ptr(w), N, K, group_size, int(bool(zero_point)), _ptr(qweight), _ptr(scales),
                      _ptr(qzeros) if zero_point else None, _stream(w))
    _check(st, "awq_pack")
    return qweight, scales, (qzeros if zero_point else None)


def awq_dequant(qweight: torch.Tensor, scales: torch.Tensor, qzeros: Optional[torch.Tensor], N: int, K: int,
                group_size: int = 128, zero_point: bool = True, w_out: Optional[torch.Tensor] = None):
    """Decode a packed weight to fp16 [N, K] (test and inspection aid)."""
    lib = load_library()
    if w_out is None:
        w_out = torch.empty((N, K), dtype=torch.float16, device=qweight.device)
    st = lib.awq_dequant(_ptr(qweight), _ptr(scales), _ptr(qzeros) if zero_point else None, _ptr(w_out), N, K,
                         group_size, int(bool(zero_point)), _stream(qweight))
    _check(st, "awq_dequant")
    return w_out


def _xy(x: torch.Tensor, N: int, y: Optional[torch.Tensor]):
    if x.dtype != torch.float16 or x.dim() != 2:
        raise ValueError("x must be a 2-D float16 tensor [M, K]")
    if y is None:
        y = torch.empty((x.shape[0], N), dtype=torch.float16, device=x.device)
    return y


def awq_gemv(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, qzeros: Optional[torch.Tensor], N: int,
             K: int, group_size: int = 128, zero_point: bool = True, y: Optional[torch.Tensor] = None):
    """Single- and few-token layer Y = X . W'^T for X fp16 [M, K], 1 <= M <= 8; returns fp16 [M, N]."""
    lib = load_library()
    y = _xy(x, N, y)
    st = lib.awq_gemv(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(qzeros) if zero_point else None, _ptr(y),
                      x.shape[0], N, K, group_size, int(bool(zero_point)), _stream(x))
    _check(st, "awq_gemv")
    return y


_WORKSPACES = {}          # (device index, stream handle) -> zero-initialised uint8 tensor
_RETIRED_WORKSPACES = []  # replaced buffers, kept alive for graphs that captured their address


def gemm_workspace(nbytes: int, device=None, stream=None) -> torch.Tensor:
    """The zero-initialised awq_gemm workspace of (``device``, ``stream``), at
    least ``nbytes`` long, kept for later calls on that stream.  awq_gemm
    returns the workspace's counters to zero, so calls in one stream's order
    share it, including calls captured into a HIP graph on that stream.
    Calls on different streams get different buffers, since overlapping
    calls on one buffer would break its per-tile counters.

    Under graph capture the buffer is not created or grown (its zero fill
    would only be recorded into the graph): call once eagerly on the
    capture stream first, or pass ``workspace=`` explicitly."""
    device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    idx = device.index if device.index is not None else torch.cuda.current_device()
    if stream is None:
        stream = torch.cuda.current_stream(idx)
    key = (idx, stream.cuda_stream)
    ws = _WORKSPACES.get(key)
    if ws is None or ws.numel() < nbytes:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError(
                f"awq_gemm needs a {nbytes}-byte split-K workspace on stream {stream.cuda_stream:#x} of cuda:{idx}, "
                "and none of that size exists; a workspace cannot be created during graph capture. Make one "
                "eager call of the largest shape on the capture stream before capturing, or pass workspace= "
                "(a zero-filled uint8 tensor of awq_gemm_workspace_bytes(...) bytes)")
        if ws is not None:
            _RETIRED_WORKSPACES.append(ws)
        with torch.cuda.stream(stream):  # zero fill ordered before this stream's next call
            ws = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=torch.device("cuda", idx))
        _WORKSPACES[key] = ws
    return ws


def awq_gemm(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, qzeros: Optional[torch.Tensor], N: int,
             K: int, group_size: int = 128, zero_point: bool = True, y: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None):
    """Batched layer Y = X . W'^T for X fp16 [M, K]; returns fp16 [M, N]."""
    lib = load_library()
    y = _xy(x, N, y)
    M = x.shape[0]
    need = awq_gemm_workspace_bytes(M, N, K, group_size)
    if need and workspace is None:
        workspace = gemm_workspace(need, x.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.awq_gemm(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(qzeros) if zero_point else None, _ptr(y), M, N, K,
                      group_size, int(bool(zero_point)), _ptr(workspace), ws_bytes, _stream(x))
    _check(st, "awq_gemm")
    return y


def awq_gemm_noalloc(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, qzeros: Optional[torch.Tensor],
                     N: int, K: int, group_size: int = 128, zero_point: bool = True,
                     y: torch.Tensor = None) -> torch.Tensor:
    """awq_gemm with the library's fixed device scratch as the split-K
    workspace: the C call allocates nothing (``y`` must be passed, so that
    this wrapper allocates nothing either).  Calls that may overlap on one
    GPU share the scratch and race."""
    lib = load_library()
    if y is None:
        raise ValueError("awq_gemm_noalloc takes a preallocated output y")
    if x.dtype != torch.float16 or x.dim() != 2:
        raise ValueError("x must be a 2-D float16 tensor [M, K]")
    st = lib.awq_gemm_noalloc(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(qzeros) if zero_point else None, _ptr(y),
                              x.shape[0], N, K, group_size, int(bool(zero_point)), _stream(x))
    _check(st, "awq_gemm_noalloc")
    return y


class PackedWeight(NamedTuple):
    qweight: torch.Tensor
    scales: torch.Tensor
    qzeros: Optional[torch.Tensor]
    N: int
    K: int
    group_size: int
    zero_point: bool


def pack(W: torch.Tensor, q_group_size: int = 128, zero_point: bool = True) -> PackedWeight:
    """Quantize an ``nn.Linear`` weight [out, in] on the GPU (``quant_config``: w_bit 4)."""
    qw, sc, qz = awq_pack(W, q_group_size, zero_point)
    return PackedWeight(qw, sc, qz, W.shape[0], W.shape[1], q_group_size, bool(zero_point))


def pack_fused(weights, q_group_size: int = 128, zero_point: bool = True) -> PackedWeight:
    """Pack several weights that read the same input (e.g. the q, k and v
    projections, or gate and up) as one weight of N = sum of their N, so one
    launch computes all of them ("AI-Research-SKILLs AWQ 高级使用指南", section
    层融合: Q, K, V merged into one GEMM, gate and up fused).

    Each part is quantized by its own ``awq_pack`` call straight into its
    slice of the fused buffers: rows are independent and the scales/zero
    points are stored per octet of rows, so a part with N a multiple of 8 is a
    contiguous slice of every array and the result is bit-identical to packing
    the concatenated weight.  The output of ``linear`` is the concatenation of
    the parts' outputs, in order."""
    weights = list(weights)
    if not weights:
        raise ValueError("pack_fused needs at least one weight")
    K = weights[0].shape[1]
    if any(w.dim() != 2 or w.shape[1] != K for w in weights):
        raise ValueError("fused weights must all be [N_i, K] with the same K")
    N = sum(w.shape[0] for w in weights)
    G = K // q_group_size if q_group_size > 0 else 0
    dev = weights[0].device
    qweight = torch.empty((N, K // 8), dtype=torch.int32, device=dev)
    scales = torch.empty((N // 8, G, 8), dtype=torch.float16, device=dev)
    qzeros = torch.empty((N // 8, G), dtype=torch.int32, device=dev) if zero_point else None
    n0 = 0
    for w in weights:
        n = w.shape[0]
        if n % 8:
            raise ValueError("every fused part needs N % 8 == 0")
        awq_pack(w, q_group_size, zero_point, qweight=qweight[n0:n0 + n], scales=scales[n0 // 8:(n0 + n) // 8],
                 qzeros=qzeros[n0 // 8:(n0 + n) // 8] if zero_point else None)
        n0 += n
    return PackedWeight(qweight, scales, qzeros, N, K, q_group_size, bool(zero_point))


def linear(x: torch.Tensor, pw: PackedWeight, version: str = "auto") -> torch.Tensor:
    """Y = X . W'^T.  ``version`` "GEMV" (up to 8 tokens), "GEMM" (any batch) or "auto"."""
    x2 = x.reshape(-1, pw.K)
    v = version.upper()
    if v == "AUTO":
        v = "GEMV" if x2.shape[0] <= 8 else "GEMM"
    fn = awq_gemv if v == "GEMV" else awq_gemm
    y = fn(x2, pw.qweight, pw.scales, pw.qzeros, pw.N, pw.K, pw.group_size, pw.zero_point)
    return y.reshape(*x.shape[:-1], pw.N)


def awq_scale_candidates(x: torch.Tensor, alphas, w: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Candidate per-channel scales s[c] = max(mean |x|, 1e-4) ** alphas[c] for fp16
    calibration activations ``x`` [M, K]; with ``w`` [N, K] (duo scaling) also
    divided by max(mean |w|, 1e-4) ** (1 - alphas[c]).  Returns fp32
    [len(alphas), K] on x's device."""
    lib = load_library()
    alphas = [float(a) for a in alphas]
    M, K = x.shape
    N = w.shape[0] if w is not None else 0
    s = torch.empty((len(alphas), K), dtype=torch.float32, device=x.device)
    ws = torch.empty(max(1, int(lib.awq_scale_candidates_workspace_bytes(M, N, K))), dtype=torch.uint8,
                     device=x.device)
    arr = (ctypes.c_float * len(alphas))(*alphas)
    st = lib.awq_scale_candidates(_ptr(x), M, K, _ptr(w), N, int(w is not None), ctypes.cast(arr, ctypes.c_void_p),
                                  len(alphas), _ptr(s), _ptr(ws), ws.numel(), _stream(x))
    _check(st, "awq_scale_candidates")
    return s


def awq_scale_loss(x: torch.Tensor, w: torch.Tensor, s: torch.Tensor, group_size: int = 128,
                   zero_point: bool = True) -> torch.Tensor:
    """L(s_c) = ||Q(W s_c)(s_c^-1 X) - W X||_F for every row s_c of the fp32 ``s``
    [count, K]; ``x`` fp16 [M, K], ``w`` fp16 [N, K].  Returns fp64 [count] on the GPU."""
    lib = load_library()
    M, K = x.shape
    N = w.shape[0]
    s2 = s.reshape(-1, K)
    count = s2.shape[0]
    loss = torch.empty(count, dtype=torch.float64, device=x.device)
    ws = torch.empty(max(1, int(lib.awq_scale_loss_workspace_bytes(count, M, N, K))), dtype=torch.uint8,
                     device=x.device)
    st = lib.awq_scale_loss(_ptr(x), _ptr(w), _ptr(s2), count, M, N, K, group_size, int(bool(zero_point)), _ptr(ws),
                            ws.numel(), _ptr(loss), _stream(x))
    _check(st, "awq_scale_loss")
    return loss


DEFAULT_ALPHAS = tuple(i / 20 for i in range(20))


class ScaleSearch(NamedTuple):
    best: torch.Tensor    # int32 [1] on the device: index of the chosen candidate
    scale: torch.Tensor   # fp32 [K] on the device: the chosen s
    losses: torch.Tensor  # fp64 [count] on the device: L(s) of every candidate, in the order of alphas
    alphas: tuple

    @property
    def alpha(self) -> float:
        """The chosen exponent (reads the index back from the device)."""
        return self.alphas[int(self.best.item())]


def awq_scale_search(x: torch.Tensor, w: torch.Tensor, group_size: int = 128, zero_point: bool = True,
                     alphas=DEFAULT_ALPHAS, duo: bool = False) -> ScaleSearch:
    """Activation-aware scale search on the device: L(s) for s = a ** alpha
    (duo: a ** alpha / b ** (1 - alpha)) over ``alphas`` and the first
    candidate with the smallest loss.  ``x`` fp16 [M, K] calibration
    activations, ``w`` fp16 [N, K].  Nothing is read back to the host."""
    lib = load_library()
    alphas = tuple(float(a) for a in alphas)
    M, K = x.shape
    N = w.shape[0]
    dev = x.device
    s_best = torch.empty(K, dtype=torch.float32, device=dev)
    best = torch.empty(1, dtype=torch.int32, device=dev)
    losses = torch.empty(len(alphas), dtype=torch.float64, device=dev)
    ws = torch.empty(max(1, int(lib.awq_scale_search_workspace_bytes(len(alphas), M, N, K))), dtype=torch.uint8,
                     device=dev)
    arr = (ctypes.c_float * len(alphas))(*alphas)
    st = lib.awq_scale_search(_ptr(x), _ptr(w), M, N, K, group_size, int(bool(zero_point)),
                              ctypes.cast(arr, ctypes.c_void_p), len(alphas), int(bool(duo)), _ptr(s_best),
                              _ptr(best), _ptr(losses), _ptr(ws), ws.numel(), _stream(x))
    _check(st, "awq_scale_search")
    return ScaleSearch(best, s_best, losses, alphas)


def search_scale(x: torch.Tensor, w: torch.Tensor, group_size: int = 128, zero_point: bool = True,
                 alphas=None, duo: bool = False) -> ScaleSearch:
    """Activation-aware scale search (default grid 0, 1/20, ..., 19/20).  The
    chosen s is applied as W * s before packing and s^-1 on the activations."""
    return awq_scale_search(x, w, group_size, zero_point, DEFAULT_ALPHAS if alphas is None else alphas, duo)


def awq_scale_columns(src: torch.Tensor, s: torch.Tensor, divide: bool = False,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """fp16(src * s) per input channel (or fp16(src / s) with ``divide``)."""
    lib = load_library()
    rows, K = src.shape
    if out is None:
        out = torch.empty_like(src)
    st = lib.awq_scale_columns(_ptr(src), rows, K, _ptr(s), int(bool(divide)), _ptr(out), _stream(src))
    _check(st, "awq_scale_columns")
    return out


DEFAULT_CLIP_RATIOS = tuple(1.0 - 0.025 * i for i in range(20))


def awq_clip_search(x: torch.Tensor, w: torch.Tensor, group_size: int = 128, zero_point: bool = True,
                    ratios=DEFAULT_CLIP_RATIOS):
    """Weight clipping: per group, the ratio in ``ratios`` with the smallest
    output error over ``x``.  Returns (clipped fp16 weights [N, K], chosen
    ratio index int32 [N, K / group_size])."""
    lib = load_library()
    M, K = x.shape
    N = w.shape[0]
    ratios = [float(r) for r in ratios]
    out = torch.empty_like(w)
    choice = torch.empty((N, K // group_size), dtype=torch.int32, device=w.device)
    ws = torch.empty(max(1, int(lib.awq_clip_search_workspace_bytes(len(ratios), M, N, K, group_size))),
                     dtype=torch.uint8, device=w.device)
    arr = (ctypes.c_float * len(ratios))(*ratios)
    st = lib.awq_clip_search(_ptr(x), _ptr(w), M, N, K, group_size, int(bool(zero_point)),
                             ctypes.cast(arr, ctypes.c_void_p), len(ratios), _ptr(out), _ptr(choice), _ptr(ws),
                             ws.numel(), _stream(x))
    _check(st, "awq_clip_search")
    return out, choice


class QuantizedLinear(NamedTuple):
    packed: PackedWeight
    input_scale: torch.Tensor  # fp32 [K]: the layer computes on fp16(x / input_scale)
    search: ScaleSearch        # the scale search (chosen index and losses stay on the device)


def quantize_awq(w: torch.Tensor, x: torch.Tensor, q_group_size: int = 128, zero_point: bool = True,
                 alphas=None, clip_ratios=DEFAULT_CLIP_RATIOS, apply_clip: bool = True,
                 duo_scaling: bool = False) -> QuantizedLinear:
    """The activation-aware quantization of one linear layer from calibration
    activations ``x`` [M, K]: scale search (the candidate s with the smallest
    L(s)), weights scaled by s, optional clipping search on the scaled layer,
    then packing; every step on the device, with no host synchronization.
    The packed layer expects activations divided by ``input_scale``
    (``awq_scale_columns(x, s, divide=True)``, or folded into the producer of x)."""
    res = search_scale(x, w, q_group_size, zero_point, alphas, duo_scaling)
    ws = awq_scale_columns(w, res.scale)
    if apply_clip:
        xs = awq_scale_columns(x, res.scale, divide=True)
        ws, _ = awq_clip_search(xs, ws, q_group_size, zero_point, clip_ratios)
    return QuantizedLinear(pack(ws, q_group_size, zero_point), res.scale, res)


# The calls below serve single tokens, where the kernel takes a few microseconds and the binding counts: one library
# call each, the checks on attributes only, the stream's handle without its Python object where torch offers that.
_F16, _F32, _I32 = torch.float16, torch.float32, torch.int32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _handle(t: torch.Tensor) -> int:
    """The handle of the current stream of a GPU tensor's device."""
    return _raw_stream(t.get_device()) if _raw_stream is not None else _stream(t)


def _rows2d(t: torch.Tensor, rows: Optional[int], width: int, what: str):
    """(address, row stride) of a float16 matrix on the GPU whose rows are contiguous and do not overlap."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not _F16 or len(shape) != 2 or shape[1] != width or (rows is not None and shape[0] != rows):
        raise ValueError(f"{what} must be a float16 tensor [{'rows' if rows is None else rows}, {width}]")
    if not t.is_cuda:
        raise ValueError("tensors passed to the AWQ kernels must live on the GPU")
    ld = stride[0] if shape[0] > 1 else width
    if (stride[1] != 1 and width > 1) or ld < width:
        raise ValueError(f"{what} must have contiguous rows that do not overlap")
    return t.data_ptr(), ld


def _flat(t: Optional[torch.Tensor], shape, dtype, what: str) -> Optional[int]:
    """Address of a contiguous GPU tensor of a given shape and type (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what} must be a {str(dtype).split('.')[-1]} tensor of shape {tuple(shape)}")
    return _ptr(t)


def _activation(name: str) -> int:
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}; got {name!r}") from None


def _with_workspace(call, need, where: str, workspace: Optional[torch.Tensor], t: torch.Tensor) -> None:
    """``call(address, bytes)`` with the caller's workspace, or else with ``need()`` bytes beside ``t`` for this call
    only.  (Its two launches hand partial sums on in them, so calls of several host threads on one stream must not
    share them; and a buffer kept for the stream would grow with the largest batch and stay.  Under graph capture the
    bytes come from the graph's own memory.)"""
    if workspace is None:
        nbytes = need()
        ws = t.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
        st = call(None if ws is None else ws.data_ptr(), nbytes)
    else:
        st = call(_ptr(workspace), workspace.numel() * workspace.element_size())
    if st != AWQ_OK:
        raise AwqError(st, where)


@functools.lru_cache(maxsize=4096)
def _bytes_of(name: str, *shape) -> int:
    """The library's workspace size of a shape: a function of its numbers alone, asked once."""
    return int(getattr(_lib or load_library(), name + "_workspace_bytes")(*shape))


def linear_fused(x: torch.Tensor, pw: PackedWeight, bias: Optional[torch.Tensor] = None, activation: str = "none",
                 gated: bool = False, residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """act(x . W'^T + bias) + residual for fp16 ``x`` [..., K], in one call.  With ``gated`` the first half of
    ``pw``'s rows is the gate (``pack_fused([gate, up])``): act(gate) * up, half as many columns.  ``x``,
    ``residual`` and ``y`` may be 2-D views with a row stride (a multiple of 8 elements); ``y`` may be
    ``residual`` itself.  One rounding to fp16.  No tokens give an empty result, here and in the calls below."""
    lib = _lib or load_library()
    qweight, scales, qzeros, N, K, group_size, zero_point = pw
    if x.dim() != 2 and x.shape[-1:] != (K,):
        raise ValueError(f"x must be a float16 tensor [..., {K}]")
    x2 = x if x.dim() == 2 else x.reshape(-1, K)
    M, width = x2.shape[0], N // 2 if gated else N
    xp, ldx = _rows2d(x2, None, K, "x")
    act = _activation(activation)
    rp, ldr = None, 0
    if residual is not None:
        r2 = residual
        if residual.dim() != 2:
            if residual.shape != (*x.shape[:-1], width):
                raise ValueError(f"residual must be a float16 tensor {[*x.shape[:-1], width]}")
            r2 = residual.reshape(-1, width)
        rp, ldr = _rows2d(r2, M, width, "residual")
    if y is None:
        out = x2.new_empty((M, width))
        yp, ldy = out.data_ptr(), width
    else:
        out = y
        yp, ldy = _rows2d(y, M, width, "y")
    bp = _flat(bias, (N,), _F16, "bias")
    qp, sp, zp = _ptr(qweight), _ptr(scales), _ptr(qzeros) if zero_point else None
    stream = _handle(x2)
    if M > 0:
        _with_workspace(
            lambda ws, n: lib.awq_linear_fused(xp, ldx, qp, sp, zp, bp, act, gated, rp, ldr, yp, ldy, M, N, K,
                                               group_size, zero_point, ws, n, stream),
            lambda: _bytes_of("awq_linear_fused", M, N, K, group_size, gated), "awq_linear_fused", workspace, x2)
    return out if y is not None or x.dim() == 2 else out.reshape(*x.shape[:-1], width)


def mlp(x: torch.Tensor, gate_up: PackedWeight, down: PackedWeight, activation: str = "silu",
        residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A decoder block's gated MLP, down(act(gate(x)) * up(x)) + residual, in two fused layers."""
    return linear_fused(linear_fused(x, gate_up, activation=activation, gated=True), down, residual=residual)


class ExpertRoute(NamedTuple):
    ids: torch.Tensor        # int32 [T, top_k]: each slot's expert, -1 for none
    weights: torch.Tensor    # fp32 [T, top_k]
    offsets: torch.Tensor    # int32 [E + 1]: expert e's rows are offsets[e] .. offsets[e + 1] - 1
    rows: torch.Tensor       # int32 [T * top_k]: the slot t * top_k + j of each row, -1 past offsets[E]
    positions: torch.Tensor  # int32 [T, top_k]: each slot's row, -1 for none


def route_experts(logits: torch.Tensor, top_k: int, renormalize: bool = True,
                  workspace: Optional[torch.Tensor] = None) -> ExpertRoute:
    """The ``top_k`` largest of each token's expert logits (fp16 or fp32 [T, E]; the lower index first among equal
    ones), their softmax weights (over the chosen ones, or over all E without ``renormalize``), and the tokens'
    slots sorted by expert.  Logits of -inf or NaN are masked; a slot left without an expert has id -1."""
    lib = _lib or load_library()
    wide = logits.dtype is _F32
    if logits.dim() != 2 or not (wide or logits.dtype is _F16):
        raise ValueError("logits must be a 2-D float16 or float32 tensor [T, E]")
    if not logits.is_cuda:
        raise ValueError("tensors passed to the AWQ kernels must live on the GPU")
    T, E = logits.shape
    ld, inner = logits.stride()
    if T == 1:
        ld = E
    if inner != 1 and E > 1:
        raise ValueError("logits must have contiguous rows")
    if not 1 <= top_k <= min(E, 64):
        raise AwqError(AWQ_ERR_OPTION, "awq_route_experts")
    if logits.data_ptr() % 16:  # a view that begins inside a 16-byte unit: the library takes aligned buffers
        logits = logits.clone(memory_format=torch.contiguous_format)
        ld = E
    shape = (T, top_k)
    ids = logits.new_empty(shape, dtype=_I32)
    weights = logits.new_empty(shape, dtype=_F32)
    offsets = logits.new_empty(E + 1, dtype=_I32)
    rows = logits.new_empty(T * top_k, dtype=_I32)
    positions = logits.new_empty(shape, dtype=_I32)
    if T == 0:
        return ExpertRoute(ids, weights, offsets.zero_(), rows, positions)
    need = lib.awq_route_experts_workspace_bytes(T, E) if workspace is None else 0
    if need:
        workspace = logits.new_empty(need, dtype=torch.uint8)
    st = lib.awq_route_experts(logits.data_ptr(), ld, wide, T, E, top_k, renormalize, ids.data_ptr(),
                               weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(), positions.data_ptr(),
                               _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
                               _handle(logits))
    _check(st, "awq_route_experts")
    return ExpertRoute(ids, weights, offsets, rows, positions)


class PackedExperts(NamedTuple):
    qweight: torch.Tensor            # int32 [E, N, K / 8]
    scales: torch.Tensor             # fp16 [E, N / 8, G, 8]
    qzeros: Optional[torch.Tensor]   # int32 [E, N / 8, G]
    E: int
    N: int
    K: int
    group_size: int
    zero_point: bool


_PACK_ROWS = 1 << 21  # most rows of one awq_pack call


def pack_experts(W, q_group_size: int = 128, zero_point: bool = True) -> PackedExperts:
    """Quantize the experts' weights [E, out, in] (a tensor, or a list of [out, in]).  Expert by expert the same
    bits as ``pack``: rows are independent and octets of them do not cross experts, so the rows of as many experts
    as one call takes are one tall weight to ``awq_pack``."""
    W = W if isinstance(W, torch.Tensor) else torch.stack(list(W))
    if W.dtype != torch.float16 or W.dim() != 3:
        raise ValueError("W must be a 3-D float16 tensor [E, N, K]")
    E, N, K = W.shape
    if N % 8:
        raise AwqError(AWQ_ERR_SHAPE, "awq_pack")
    G = K // q_group_size if q_group_size > 0 else 0
    qweight = torch.empty((E, N, K // 8), dtype=torch.int32, device=W.device)
    scales = torch.empty((E, N // 8, G, 8), dtype=torch.float16, device=W.device)
    qzeros = torch.empty((E, N // 8, G), dtype=torch.int32, device=W.device) if zero_point else None
    step = max(1, _PACK_ROWS // max(N, 1))
    for e in range(0, E, step):
        part = slice(e, min(e + step, E))
        own = qzeros[part] if zero_point else None
        if zero_point and own.data_ptr() % 16:  # awq_pack writes whole aligned buffers: through one, then in place
            own = torch.empty_like(own)
        awq_pack(W[part].flatten(0, 1), q_group_size, zero_point, qweight[part], scales[part], own)
        if zero_point and own.data_ptr() != qzeros[part].data_ptr():
            qzeros[part] = own
    return PackedExperts(qweight, scales, qzeros, E, N, K, q_group_size, bool(zero_point))


def linear_experts(x: torch.Tensor, pe: PackedExperts, route: ExpertRoute, bias: Optional[torch.Tensor] = None,
                   activation: str = "none", gated: bool = False, y: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Every routed slot's token (fp16 ``x`` [T, K]) through its expert's layer and epilogue (``bias`` [E, N],
    ``gated`` as in ``linear_fused``): fp16 [T * top_k, N or N / 2], rows sorted by expert as ``route.rows`` says.
    Rows before ``route.offsets[0]`` or past ``route.offsets[E]`` (slots without an expert, or with one outside the
    slice of a route's experts that ``route.offsets[e0:e1 + 1]`` names) are not written."""
    lib = _lib or load_library()
    qweight, scales, qzeros, E, N, K, group_size, zero_point = pe
    T, top_k = route.ids.shape
    R, width = T * top_k, N // 2 if gated else N
    op = _flat(route.offsets, (E + 1,), _I32, "route.offsets")
    wp = _flat(route.rows, (R,), _I32, "route.rows")
    xp, ldx = _rows2d(x, T, K, "x")
    act = _activation(activation)
    if y is None:
        out = x.new_empty((R, width))
        yp, ldy = out.data_ptr(), width
    else:
        out = y
        yp, ldy = _rows2d(y, R, width, "y")
    bp = _flat(bias, (E, N), _F16, "bias")
    qp, sp, zp = _ptr(qweight), _ptr(scales), _ptr(qzeros) if zero_point else None
    stream = _handle(x)
    if R > 0:
        _with_workspace(
            lambda ws, n: lib.awq_linear_experts(xp, ldx, T, wp, top_k, op, R, E, qp, sp, zp, bp, act, gated, yp, ldy, N,
                                                 K, group_size, zero_point, ws, n, stream),
            lambda: _bytes_of("awq_linear_experts", R, E, N, K, group_size, gated), "awq_linear_experts", workspace, x)
    return out


def combine_experts(h: torch.Tensor, pe: PackedExperts, route: ExpertRoute, bias: Optional[torch.Tensor] = None,
                    residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The experts' second layer on the sorted rows ``h`` [T * top_k, K] and each token's weighted sum, plus
    ``residual`` [T, N]: fp16 [T, N], one rounding.  With a slice of the route's offsets, the sum over the slice
    (of at least ``top_k`` experts)."""
    lib = _lib or load_library()
    qweight, scales, qzeros, E, N, K, group_size, zero_point = pe
    T, top_k = shape = route.ids.shape
    op = _flat(route.offsets, (E + 1,), _I32, "route.offsets")
    pp = _flat(route.positions, shape, _I32, "route.positions")
    wp = _flat(route.weights, shape, _F32, "route.weights")
    hp, ldh = _rows2d(h, T * top_k, K, "h")
    rp, ldr = (None, 0) if residual is None else _rows2d(residual, T, N, "residual")
    if y is None:
        out = h.new_empty((T, N))
        yp, ldy = out.data_ptr(), N
    else:
        out = y
        yp, ldy = _rows2d(y, T, N, "y")
    bp = _flat(bias, (E, N), _F16, "bias")
    qp, sp, zp = _ptr(qweight), _ptr(scales), _ptr(qzeros) if zero_point else None
    stream = _handle(h)
    if T > 0:
        _with_workspace(
            lambda ws, n: lib.awq_combine_experts(hp, ldh, op, pp, wp, T, top_k, E, qp, sp, zp, bp, rp, ldr, yp, ldy, N,
                                                  K, group_size, zero_point, ws, n, stream),
            lambda: _bytes_of("awq_combine_experts", T, top_k, E, N, K, group_size), "awq_combine_experts", workspace, h)
    return out


def expert_mlp(x: torch.Tensor, logits: torch.Tensor, gate_up: PackedExperts, down: PackedExperts, top_k: int,
               activation: str = "silu", renormalize: bool = True,
               residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A mixture-of-experts MLP: route each token of ``x`` [T, K] by its ``logits`` [T, E], the experts' gated first
    layers, their second layers weighted and added up, plus ``residual``.  Nothing is read back to the host."""
    route = route_experts(logits, top_k, renormalize)
    h = linear_experts(x, gate_up, route, activation=activation, gated=True)
    return combine_experts(h, down, route, residual=residual)


class KvCache(NamedTuple):
    k: torch.Tensor                 # fp16 [pages, kv_heads, page_size, head_dim]
    v: torch.Tensor
    bounds: Optional[torch.Tensor]  # fp16 [pages, kv_heads, 2, head_dim]: each page's least and greatest key


class Sequences(NamedTuple):
    offsets: torch.Tensor  # int32 [B + 1]: sequence b's new tokens are rows offsets[b] .. offsets[b + 1] - 1
    lengths: torch.Tensor  # int32 [B]: its tokens, the new ones among them
    tables: torch.Tensor   # int32 [B, width]: its pages


def kv_cache(pages: int, kv_heads: int, head_dim: int, page_size: int = 32, bounds: bool = True,
             device="cuda") -> KvCache:
    """An uninitialised cache; with ``bounds``, one that ``select_pages`` can choose from."""
    shape = (pages, kv_heads, page_size, head_dim)
    k, v = (torch.empty(shape, dtype=torch.float16, device=device) for _ in range(2))
    return KvCache(k, v, torch.empty((pages, kv_heads, 2, head_dim), dtype=torch.float16, device=device) if bounds else None)


def _beside(t: Optional[torch.Tensor], shape, dtype, device: int, what: str) -> Optional[int]:
    """Address of a contiguous tensor of a given shape and type on the GPU of the rows (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what} must be a {str(dtype).split('.')[-1]} tensor of shape {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{what} must live on the GPU of the rows")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _int32(value: int, where: str) -> int:
    """A number for the library as it is: the call would pass on its lowest 32 bits."""
    if not -1 << 31 <= value < 1 << 31:
        raise AwqError(AWQ_ERR_OPTION, where)
    return value


def _cache_shape(cache: KvCache):
    """(pages, key heads, page size, head size) of a cache; it may be without pages where there are no tokens."""
    shape = cache.k.shape
    if len(shape) != 4 or 0 in shape[1:] or cache.v.shape != shape:
        raise ValueError("the cache's keys and values must be float16 tensors [pages, kv_heads, page_size, head_dim]")
    return shape


def _cache_call(x: torch.Tensor, cache: KvCache, seqs: Sequences, extra: int, what: str):
    """(device, row address, row stride, the batch's arguments, those of the pages) of rows ``x`` that hold ``extra``
    vectors per key head beside the queries' (keys and values); everything on the rows' device, which is the current
    one for the call."""
    k, v, bounds = cache
    offsets, lengths, tables = seqs
    pages, kv_heads, page_size, dim = shape = _cache_shape(cache)
    if x.dim() != 2 or x.shape[1] % dim:
        raise ValueError(f"{what} must be a float16 tensor [T, heads * {dim}]")
    T, width = x.shape
    heads = width // dim - extra * kv_heads
    if heads < 1 or heads % kv_heads:
        raise ValueError(f"{what} must hold a multiple of {kv_heads} query heads")
    xp, ldx = _rows2d(x, None, width, what)
    if lengths.dim() != 1 or tables.dim() != 2:
        raise ValueError("seqs.lengths must be an int32 tensor [B], seqs.tables one [B, width]")
    B, device = lengths.shape[0], x.get_device()
    columns = tables.shape[1]
    batch = (_beside(offsets, (B + 1,), _I32, device, "seqs.offsets"),
             _beside(lengths, (B,), _I32, device, "seqs.lengths"),
             _beside(tables, (B, columns), _I32, device, "seqs.tables"), columns, T, B, heads, kv_heads, dim)
    return device, xp, ldx, batch, (_beside(k, shape, _F16, device, "cache.k"),
                                    _beside(v, shape, _F16, device, "cache.v"), pages, page_size)


def _page_bounds(cache: KvCache, device: int) -> Optional[int]:
    pages, kv_heads, _, dim = cache.k.shape
    return _beside(cache.bounds, (pages, kv_heads, 2, dim), _F16, device, "cache.bounds")


def _workspace_beside(workspace: Optional[torch.Tensor], device: int) -> None:
    if workspace is not None and workspace.get_device() != device:
        raise ValueError("workspace must live on the GPU of the rows")


def _output(y: Optional[torch.Tensor], x: torch.Tensor, width: int, what: str):
    if y is None:
        out = x.new_empty((x.shape[0], width))
        return out, out.data_ptr(), width
    if y.get_device() != x.get_device():
        raise ValueError(f"{what} must live on the GPU of the rows")
    return (y, *_rows2d(y, x.shape[0], width, what))


def append_kv(qkv: torch.Tensor, cache: KvCache, seqs: Sequences, inv_freq: Optional[torch.Tensor] = None,
              positions: Optional[torch.Tensor] = None, axes: Optional[torch.Tensor] = None, interleaved: bool = False,
              q: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The new tokens' rows ``qkv`` [T, (q_heads + 2 kv_heads) * head_dim] of a fused q/k/v layer: keys (rotated) and
    values into the cache's pages, the pages' bounds kept up to date if it has them; returns the rotated queries
    [T, q_heads * head_dim].  ``inv_freq`` (fp32 [R / 2]): pair i of the first R channels turns by position *
    inv_freq[i]; None: no rotation.  ``positions`` int32 [T] or [T, axes]: None takes each token's place in its
    sequence.  With several axes ``axes`` (int32 [R / 2]) says which one pair i turns by.  Pairs are channels
    (i, R / 2 + i), or (2 i, 2 i + 1) with ``interleaved``.  ``q`` may be the queries' columns of ``qkv``; its rows of
    tokens without a place (behind the last sequence) are left as they are, uninitialised in a new one.  A page's bounds
    only grow until its first slot is written again."""
    lib = _lib or load_library()
    device, xp, ldx, batch, (kp, vp, pages, page_size) = _cache_call(qkv, cache, seqs, 2, "qkv")
    bp = _page_bounds(cache, device)
    width = batch[6] * batch[8]
    out, qp, ldq = _output(q, qkv, width, "q")
    T, count = qkv.shape[0], 1
    half = 0 if inv_freq is None else inv_freq.shape[0]
    shape = (T,)
    if positions is not None and positions.dim() == 2:
        shape = (T, count := positions.shape[1])
    fp = _beside(inv_freq, (half,), _F32, device, "inv_freq")
    pp = _beside(positions, shape, _I32, device, "positions")
    ap = _beside(axes, (half,), _I32, device, "axes")
    if T > 0:
        with _device_of(device):
            st = lib.awq_append_kv(xp, ldx, *batch, fp, 2 * half, interleaved, pp, count, ap, qp, ldq, kp, vp, bp, pages,
                                   page_size, _handle(qkv))
        _check(st, "awq_append_kv")
    return out


class _Here:
    def __enter__(self):
        return None

    def __exit__(self, *_):
        return False


_HERE = _Here()


def _device_of(device: int):
    """The device as the current one, for a launch; nothing to do where it is already."""
    return _HERE if device == torch.cuda.current_device() else torch.cuda.device(device)


def _attend_rows(name: str, q, cache, seqs, scale, y, workspace, options, shape):
    """awq_attend and awq_attend_pages: ``options`` between the scale and the pages, ``shape`` of the workspace."""
    lib = _lib or load_library()
    device, qp, ldq, batch, (kp, vp, pages, page_size) = _cache_call(q, cache, seqs, 0, "q")
    _workspace_beside(workspace, device)
    out, yp, ldy = _output(y, q, q.shape[1], "y")
    if scale is None:
        scale = batch[8] ** -0.5
    if q.shape[0] > 0:
        call, stream = getattr(lib, name), _handle(q)
        with _device_of(device):
            _with_workspace(
                lambda ws, n: call(qp, ldq, *batch, scale, *options, kp, vp, pages, page_size, yp, ldy, ws, n, stream),
                lambda: _bytes_of(name, *shape(batch, page_size)), name, workspace, q)
    return out


def attend(q: torch.Tensor, cache: KvCache, seqs: Sequences, scale: Optional[float] = None, shared: int = 0,
           y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention of the new tokens' queries ``q`` [T, q_heads * head_dim] over their sequences' pages (their own
    keys appended already): fp16 [T, q_heads * head_dim].  ``scale``: head_dim ** -0.5 by default.  ``shared``: how many
    tokens all sequences begin with (a multiple of the page size); their pages, those of the table of the first
    sequence that has rows, are read and multiplied once for the whole batch (a new token among them sees those
    up to its own place).  A row without keys gives 0; rows of no sequence are left as they are."""
    _int32(shared, "awq_attend")
    return _attend_rows("awq_attend", q, cache, seqs, scale, y, workspace, (shared,),
                        lambda b, size: (b[4], b[5], b[6], b[7], b[8], b[3], size, shared))


def select_pages(q: torch.Tensor, cache: KvCache, seqs: Sequences, count: int, first: int = 1, recent: int = 1,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """For each new token and key head the pages of its sequence to attend to, int32 [T, kv_heads, count], ascending,
    -1 past the last: all of them up to the token's place if they are at most ``count``, or else the ``first`` first,
    the ``recent`` last, and those between whose bounds allow the largest products with the queries."""
    lib = _lib or load_library()
    for n in (count, first, recent):
        _int32(n, "awq_select_pages")
    device, qp, ldq, batch, (_, _, pages, page_size) = _cache_call(q, cache, seqs, 0, "q")
    _workspace_beside(workspace, device)
    if cache.bounds is None:
        raise ValueError("select_pages needs a cache with bounds")
    bp = _page_bounds(cache, device)
    if count < 1:
        raise AwqError(AWQ_ERR_OPTION, "awq_select_pages")
    T, kv_heads = q.shape[0], batch[7]
    out = q.new_empty((T, kv_heads, count), dtype=_I32)
    if T > 0:
        stream = _handle(q)
        with _device_of(device):
            _with_workspace(
                lambda ws, n: lib.awq_select_pages(qp, ldq, *batch, bp, pages, page_size, count, first, recent,
                                                   out.data_ptr(), ws, n, stream),
                lambda: _bytes_of("awq_select_pages", T, kv_heads, batch[3], count), "awq_select_pages", workspace, q)
    return out


def attend_pages(q: torch.Tensor, cache: KvCache, seqs: Sequences, pages: torch.Tensor, scale: Optional[float] = None,
                 y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``attend`` over chosen pages only (``select_pages``' int32 [T, kv_heads, count], or any such choice of a
    sequence's pages: each at most once, negative ones last), up to each token's place."""
    if q.dim() != 2 or pages.dim() != 3 or pages.shape[:2] != (q.shape[0], _cache_shape(cache)[1]):
        raise ValueError("pages must be an int32 tensor [T, kv_heads, count]")
    count = pages.shape[2]
    return _attend_rows("awq_attend_pages", q, cache, seqs, scale, y, workspace,
                        (_beside(pages, pages.shape, _I32, q.get_device(), "pages"), count),
                        lambda b, size: (b[4], b[6], b[7], b[8], size, count))


def _check_attention(x, qkv, o, cache, seqs, residual, scale, shared, pages, first, recent) -> None:
    """What the calls of `attention` behind `append_kv` would refuse, before that writes to the cache."""
    if pages and shared:
        raise ValueError("chosen pages are of each sequence's own table: with pages, shared must be 0")
    _, kv_heads, page_size, dim = _cache_shape(cache)
    if x.dim() != 2 or seqs.tables.dim() != 2 or seqs.lengths.dim() != 1:
        raise ValueError("x must be a float16 tensor [T, K], seqs.lengths an int32 tensor [B], seqs.tables one [B, width]")
    T, width, heads = x.shape[0], seqs.tables.shape[1], qkv.N // dim - 2 * kv_heads
    if heads < 1 or heads % kv_heads or qkv.N % dim or o.K != heads * dim:
        raise ValueError(f"qkv must give a multiple of {kv_heads} query heads and {2 * kv_heads} others of {dim} channels "
                         f"each, and o take the query heads' channels; they are of {qkv.N} and {o.K}")
    if residual is not None:
        rp, ldr = _rows2d(residual, T, o.N, "residual")
        if ldr % 8 or rp % 16:
            raise AwqError(AWQ_ERR_SHAPE if ldr % 8 else AWQ_ERR_ALIGN, "awq_linear_fused")
    f32 = lambda v: ctypes.c_float(v).value  # noqa: E731
    if scale is not None and not (f32(scale) > 0.0 and f32(scale * 1.4426950408889634) < float("inf")):
        raise AwqError(AWQ_ERR_OPTION, "awq_attend")
    if pages:
        if cache.bounds is None:
            raise ValueError("attention to chosen pages needs a cache with bounds")
        _page_bounds(cache, x.get_device())
        rows, places = T * kv_heads, pages * page_size
        if rows >= 1 << 22:
            raise AwqError(AWQ_ERR_SHAPE, "awq_select_pages")
        if pages < 1 or first < 0 or recent < 1 or first + recent > pages or rows * pages >= 1 << 31:
            raise AwqError(AWQ_ERR_OPTION, "awq_select_pages")
        if places > 1 << 30 or rows * -(-(heads // kv_heads) // 16) * (places // 32 + 1) >= 1 << 30:
            raise AwqError(AWQ_ERR_OPTION, "awq_attend_pages")
    elif shared:
        if shared < 0 or shared % page_size or shared // page_size > width:
            raise AwqError(AWQ_ERR_OPTION, "awq_attend")
        # (no workspace: not a shape that is taken, where shared keys always have parts to join)
        if T > 0 and not _bytes_of("awq_attend", T, seqs.lengths.shape[0], heads, kv_heads, dim, width, page_size, shared):
            raise AwqError(AWQ_ERR_SHAPE, "awq_attend")


def attention(x: torch.Tensor, qkv: PackedWeight, o: PackedWeight, cache: KvCache, seqs: Sequences,
              inv_freq: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
              residual: Optional[torch.Tensor] = None, scale: Optional[float] = None, shared: int = 0,
              pages: int = 0, first: int = 1, recent: int = 1, positions: Optional[torch.Tensor] = None,
              axes: Optional[torch.Tensor] = None, interleaved: bool = False) -> torch.Tensor:
    """A decoder block's attention for new tokens ``x`` [T, K]: the fused q/k/v layer (``pack_fused([q, k, v])``,
    ``bias`` its own), the tokens' keys and values appended, attention over the cache, the output layer, plus
    ``residual``.  With ``pages`` above 0 each token attends to that many pages only (``select_pages``); these come from
    the token's own table, so ``shared`` must be 0.  Nothing is written if a call is refused.  Rows of no sequence come
    back as anything."""
    _check_attention(x, qkv, o, cache, seqs, residual, scale, shared, pages, first, recent)
    rows = linear_fused(x, qkv, bias=bias)
    q = append_kv(rows, cache, seqs, inv_freq, positions, axes, interleaved)
    if pages:
        y = attend_pages(q, cache, seqs, select_pages(q, cache, seqs, pages, first, recent), scale)
    else:
        y = attend(q, cache, seqs, scale, shared)
    return linear_fused(y, o, residual=residual)
