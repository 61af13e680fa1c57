"""GPTQ layer-wise weight quantizer for NVIDIA B200 -- Python binding.

Every function named ``gptq_*`` here marshals torch tensors into the C entry
point of the same name in ``libgptq_b200.so`` (declared in include/gptq.h)
and raises ``GptqError`` on a non-OK status.  All the arithmetic runs in the
library's CUDA kernels; PyTorch only provides device memory and streams.

``quantize_linear`` chains the calls for one linear layer, the way the page
"GPTQ, with the code open" describes the method: H from the calibration
inputs, the Cholesky factor of the damped inverse, the column sweep, packed
codes.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses

import torch

from . import _lib
from ._lib import (GPTQ_BF16, GPTQ_F32, GPTQ_OP_CHOLESKY, GPTQ_OP_DEQUANT_MATVEC, GPTQ_OP_HESSIAN,
                   GPTQ_OP_QUANTIZE, GptqConfig, GptqLora)

__all__ = ["GptqError", "GptqConfig", "LayerPipeline", "gptq_workspace_size",
           "gptq_hadamard_rows", "gptq_hadamard_cols", "gptq_hessian_accumulate",
           "gptq_cholesky_inverse", "gptq_quantize_layer", "gptq_pack_int4", "gptq_pack_int3",
           "gptq_dequant", "gptq_dequant_matvec", "gptq_gather_columns_u8", "gptq_status_string",
           "make_config", "gptq_set_wait_gate", "gptq_launch_count",
           "QuantizedLinear", "LowRankAdapters", "AdaptedLinear", "gptq_lora_plan",
           "gptq_lora_apply", "gptq_lora_backward", "gptq_quantize_act8", "gptq_dequant_act8",
           "quantize_linear", "LayerQuantizer", "library"]


class GptqError(RuntimeError):
    pass


def library() -> ctypes.CDLL:
    return _lib.load()


def debug_library() -> ctypes.CDLL:
    """libgptq_b200_debug.so: the same entry points with device-side checks
    of caller-supplied indices (build it with ``build(debug=True)``)."""
    return _lib.load(_lib.DEBUG_LIB_PATH)


def gptq_device_checks(lib: ctypes.CDLL | None = None) -> int:
    """The index checks that failed since the last read, as a bit set (1: a
    group index out of range, 2: a permutation entry out of range), then
    cleared; waits for the device.  Debug library only."""
    lib = debug_library() if lib is None else lib
    flags = ctypes.c_uint32(0)
    _check(lib.gptq_device_checks(ctypes.byref(flags)), "gptq_device_checks")
    return int(flags.value)


def gptq_status_string(status: int) -> str:
    return library().gptq_status_string(int(status)).decode()


def gptq_launch_count() -> int:
    """Kernels the library has enqueued in this process so far."""
    return int(library().gptq_launch_count())


def gptq_set_wait_gate(gate: torch.Tensor | None, limit_ns: int = 1_000_000_000) -> None:
    """Test hook of the bounded device waits (see include/gptq.h): with a
    device int32 ``gate`` holding 0, the tensor-core kernels this thread
    enqueues next wait for it and give up after ``limit_ns``; None restores
    the normal behaviour."""
    if gate is not None:
        _need_cuda(gate)
        if gate.dtype != torch.int32:
            raise GptqError("gate must be a device int32 tensor")
    _check(library().gptq_set_wait_gate(_p(gate), int(limit_ns)), "gptq_set_wait_gate")


def _check(status: int, what: str) -> None:
    if status != 0:
        raise GptqError(f"{what}: {gptq_status_string(status)} (status {status})")


def _p(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _side(side_stream) -> int | None:
    """A second stream for look-ahead, or None (one stream)."""
    return None if side_stream is None else side_stream.cuda_stream


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return GPTQ_BF16
    if dt == torch.float32:
        return GPTQ_F32
    raise GptqError(f"unsupported dtype {dt} (bf16 or fp32)")


def _need_cuda(*ts) -> None:
    for t in ts:
        if t is not None and not t.is_cuda:
            raise GptqError("tensors must live on the GPU")


def make_config(bits=4, group_size=128, percdamp=0.01, actorder=False, block=128,
                sym=False) -> GptqConfig:
    return GptqConfig(int(bits), int(group_size), float(percdamp), int(block), int(bool(actorder)),
                      int(bool(sym)))


def gptq_workspace_size(op: int, rows: int, n: int, ntok: int = 0,
                        xdtype: torch.dtype = torch.bfloat16, cfg: GptqConfig | None = None) -> int:
    out = ctypes.c_size_t(0)
    st = library().gptq_workspace_size(int(op), int(rows), int(n), int(ntok), _dtype_code(xdtype),
                                       ctypes.byref(cfg) if cfg is not None else None,
                                       ctypes.byref(out))
    _check(st, "gptq_workspace_size")
    return int(out.value)


def _workspace(nbytes: int, device, ws):
    if nbytes == 0:
        return ws
    if ws is not None:
        # (an expanded tensor has elements that are not there)
        if ws.device != device or not ws.is_contiguous():
            raise GptqError(f"the workspace must be a contiguous tensor on {device}")
        if ws.numel() >= nbytes:
            return ws
    return torch.empty(nbytes + 256, dtype=torch.uint8, device=device)


def _aligned_ptr(ws) -> tuple[int | None, int]:
    if ws is None:
        return None, 0
    p = ws.data_ptr()
    off = (-p) % 256
    return p + off, ws.numel() - off


def gptq_hessian_accumulate(H: torch.Tensor, X: torch.Tensor, alpha: float = 2.0, ws=None,
                            info: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """H += alpha * X X^T for X (n features x N tokens, bf16 or fp32); returns H."""
    _need_cuda(H, X, info)
    n, ntok = X.shape
    if H.dtype != torch.float32 or H.shape != (n, n) or not H.is_contiguous():
        raise GptqError("H must be a contiguous n x n float32 tensor")
    if X.stride(1) != 1:
        raise GptqError("X must have contiguous rows (tokens)")
    need = gptq_workspace_size(GPTQ_OP_HESSIAN, 0, n, ntok, X.dtype)
    ws = _workspace(need, X.device, ws)
    wp, wn = _aligned_ptr(ws)
    st = library().gptq_hessian_accumulate(_p(H), _p(X), _dtype_code(X.dtype), n, ntok,
                                           X.stride(0), 0, float(alpha), wp, wn, _p(info),
                                           _stream(stream))
    _check(st, "gptq_hessian_accumulate")
    return H


def gptq_cholesky_inverse(H: torch.Tensor, percdamp: float = 0.01, actorder: bool = False,
                          U=None, perm=None, dead=None, info=None, ws=None, stream=None,
                          side_stream=None):
    """Dead inputs, act-order, damping and U (upper, H'^-1 = U^T U).
    Returns (U, perm, dead, info); info is a device int32 (0 = success).
    side_stream: a second torch.cuda.Stream for the look-ahead (same result)."""
    _need_cuda(H)
    n = H.shape[0]
    dev = H.device
    U = torch.empty(n, n, dtype=torch.float32, device=dev) if U is None else U
    perm = torch.empty(n, dtype=torch.int32, device=dev) if perm is None else perm
    dead = torch.empty(n, dtype=torch.uint8, device=dev) if dead is None else dead
    info = torch.empty(1, dtype=torch.int32, device=dev) if info is None else info
    need = gptq_workspace_size(GPTQ_OP_CHOLESKY, 0, n)
    ws = _workspace(need, dev, ws)
    wp, wn = _aligned_ptr(ws)
    st = library().gptq_cholesky_inverse(_p(H), n, float(percdamp), int(bool(actorder)), _p(U),
                                         _p(perm), _p(dead), _p(info), wp, wn, _stream(stream),
                                         _side(side_stream))
    _check(st, "gptq_cholesky_inverse")
    return U, perm, dead, info


def gptq_cholesky_inverse_noalloc(H: torch.Tensor, percdamp: float, actorder: bool, U, perm,
                                  dead, info, stream=None):
    """gptq_cholesky_inverse for callers that cannot allocate device memory:
    every output buffer is the caller's and the scratch is built into the
    library (n <= 2048).  Nothing is allocated here either."""
    _need_cuda(H, U, perm, dead, info)
    n = H.shape[0]
    st = library().gptq_cholesky_inverse_noalloc(_p(H), n, float(percdamp), int(bool(actorder)),
                                                 _p(U), _p(perm), _p(dead), _p(info),
                                                 _stream(stream))
    _check(st, "gptq_cholesky_inverse_noalloc")
    return U, perm, dead, info


def gptq_quantize_layer(W: torch.Tensor, U: torch.Tensor, perm, dead, cfg: GptqConfig,
                        codes=None, scales=None, zeros=None, g_idx=None, Wq=None, row_loss=None,
                        want_g_idx: bool = True, want_wq: bool = False, want_loss: bool = False,
                        ws=None, info=None, stream=None, side_stream=None) -> dict:
    """The column sweep.  Returns dict(codes, scales, zeros, g_idx, Wq, row_loss).
    info: optional device int32 (set to 0, or -2 if a device wait gave up);
    side_stream: a second torch.cuda.Stream for the look-ahead (same result)."""
    _need_cuda(W, U, perm, dead)
    rows, n = W.shape
    if not W.is_contiguous():
        raise GptqError("W must be contiguous")
    dev = W.device
    G = 1 if cfg.group_size <= 0 else (n + cfg.group_size - 1) // cfg.group_size
    codes = torch.empty(rows, n, dtype=torch.uint8, device=dev) if codes is None else codes
    scales = torch.empty(rows, G, dtype=torch.float32, device=dev) if scales is None else scales
    zeros = torch.empty(rows, G, dtype=torch.uint8, device=dev) if zeros is None else zeros
    if g_idx is None and want_g_idx:
        g_idx = torch.empty(n, dtype=torch.int32, device=dev)
    if Wq is None and want_wq:
        Wq = torch.empty(rows, n, dtype=torch.float32, device=dev)
    if row_loss is None and want_loss:
        row_loss = torch.empty(rows, dtype=torch.float32, device=dev)
    need = gptq_workspace_size(GPTQ_OP_QUANTIZE, rows, n, 0, torch.bfloat16, cfg)
    ws = _workspace(need, dev, ws)
    wp, wn = _aligned_ptr(ws)
    st = library().gptq_quantize_layer(_p(W), _dtype_code(W.dtype), rows, n, _p(U), _p(perm),
                                       _p(dead), ctypes.byref(cfg), _p(codes), _p(scales),
                                       _p(zeros), _p(g_idx), _p(Wq), _p(row_loss), wp, wn,
                                       _p(info), _stream(stream), _side(side_stream))
    _check(st, "gptq_quantize_layer")
    return {"codes": codes, "scales": scales, "zeros": zeros, "g_idx": g_idx, "Wq": Wq,
            "row_loss": row_loss}


def gptq_pack_int4(codes: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    _need_cuda(codes)
    rows, n = codes.shape
    out = torch.empty(rows, n // 8, dtype=torch.int32, device=codes.device) if out is None else out
    _check(library().gptq_pack_int4(_p(codes), rows, n, _p(out), _stream(stream)),
           "gptq_pack_int4")
    return out


def gptq_pack_int3(codes: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    _need_cuda(codes)
    rows, n = codes.shape
    out = (torch.empty(rows, 3 * n // 32, dtype=torch.int32, device=codes.device)
           if out is None else out)
    _check(library().gptq_pack_int3(_p(codes), rows, n, _p(out), _stream(stream)),
           "gptq_pack_int3")
    return out


def gptq_dequant(packed: torch.Tensor, bits: int, n: int, scales: torch.Tensor,
                 zeros: torch.Tensor, group_size: int = -1, g_idx=None,
                 out_dtype: torch.dtype = torch.float32, out=None, stream=None) -> torch.Tensor:
    _need_cuda(packed, scales, zeros, g_idx)
    rows = packed.shape[0]
    out = torch.empty(rows, n, dtype=out_dtype, device=packed.device) if out is None else out
    st = library().gptq_dequant(_p(packed), int(bits), rows, int(n), _p(scales), _p(zeros),
                                int(group_size), scales.shape[1], _p(g_idx), _p(out),
                                _dtype_code(out.dtype), _stream(stream))
    _check(st, "gptq_dequant")
    return out


def gptq_gather_columns_u8(src: torch.Tensor, perm: torch.Tensor, out=None,
                           stream=None) -> torch.Tensor:
    """out[r][k] = src[r][perm[k]] (uint8 rows x n): codes into sweep order."""
    _need_cuda(src, perm)
    rows, n = src.shape
    out = torch.empty_like(src) if out is None else out
    _check(library().gptq_gather_columns_u8(_p(src), rows, n, _p(perm), _p(out), _stream(stream)),
           "gptq_gather_columns_u8")
    return out


def gptq_dequant_matvec(packed: torch.Tensor, bits: int, n: int, scales: torch.Tensor,
                        zeros: torch.Tensor, x: torch.Tensor, group_size: int = -1, g_idx=None,
                        perm=None, out=None, ws=None, stream=None) -> torch.Tensor:
    """y = x w_hat^T with w_hat dequantized on the fly from the packed codes.
    x: (batch, n) or (n,) bf16/fp32 on the GPU; returns (batch, rows) fp32
    (or (rows,) for a 1-D x).  perm: the codes are packed in sweep order
    (see gptq_gather_columns_u8) and column k multiplies x[perm[k]]."""
    _need_cuda(packed, scales, zeros, g_idx, perm, x)
    rows = packed.shape[0]
    x2 = x.reshape(1, -1) if x.dim() == 1 else x
    if x2.shape[1] != n or not x2.is_contiguous():
        raise GptqError("x must be a contiguous (batch, n) tensor")
    batch = x2.shape[0]
    out = torch.empty(batch, rows, dtype=torch.float32, device=packed.device) if out is None else out
    need = gptq_workspace_size(GPTQ_OP_DEQUANT_MATVEC, batch, n)
    ws = _workspace(need, packed.device, ws)
    wp, wn = _aligned_ptr(ws)
    st = library().gptq_dequant_matvec(_p(packed), int(bits), rows, int(n), _p(scales), _p(zeros),
                                       int(group_size), scales.shape[1], _p(g_idx), _p(perm),
                                       _p(x2), _dtype_code(x2.dtype), batch, _p(out), wp, wn,
                                       _stream(stream))
    _check(st, "gptq_dequant_matvec")
    return out.reshape(-1) if x.dim() == 1 else out


def _hadamard(cols: bool, x: torch.Tensor, signs: torch.Tensor, block: int, out, out_dtype,
              stream):
    _need_cuda(x, signs)
    if x.dim() != 2 or x.stride(1) != 1:
        raise GptqError("x must be a 2-D tensor with contiguous rows")
    if signs.dtype != torch.float32 or not signs.is_contiguous():
        raise GptqError("signs must be a contiguous float32 tensor")
    a, b = x.shape
    if out is None:
        out = torch.empty(a, b, dtype=out_dtype or x.dtype, device=x.device)
    if out.dim() != 2 or out.shape != x.shape or out.stride(1) != 1:
        raise GptqError("out must match x, with contiguous rows")
    fn = library().gptq_hadamard_cols if cols else library().gptq_hadamard_rows
    st = fn(_p(x), _dtype_code(x.dtype), a, b, x.stride(0), _p(signs), int(block), _p(out),
            _dtype_code(out.dtype), out.stride(0), _stream(stream))
    _check(st, "gptq_hadamard_cols" if cols else "gptq_hadamard_rows")
    return out


def gptq_hadamard_rows(W: torch.Tensor, signs: torch.Tensor, block: int = 1024, out=None,
                       out_dtype=None, stream=None) -> torch.Tensor:
    """W' = W R^T with R = blockdiag(H_b / sqrt(b)) diag(signs), along the rows
    of W (rows x n).  out may be W itself (in place)."""
    return _hadamard(False, W, signs, block, out, out_dtype, stream)


def gptq_hadamard_cols(X: torch.Tensor, signs: torch.Tensor, block: int = 1024, out=None,
                       out_dtype=None, stream=None) -> torch.Tensor:
    """X' = R X along the first axis of X (n x ntok).  out may be X itself."""
    return _hadamard(True, X, signs, block, out, out_dtype, stream)


@dataclasses.dataclass
class QuantizedLinear:
    packed: torch.Tensor
    scales: torch.Tensor
    zeros: torch.Tensor
    g_idx: torch.Tensor | None
    perm: torch.Tensor
    bits: int
    group_size: int
    n: int
    codes: torch.Tensor
    info: torch.Tensor
    H: torch.Tensor | None = None
    U: torch.Tensor | None = None
    Wq: torch.Tensor | None = None
    row_loss: torch.Tensor | None = None


def quantize_linear(W: torch.Tensor, X=None, H: torch.Tensor | None = None, bits: int = 4,
                    group_size: int = 128, percdamp: float = 0.01, actorder: bool = False,
                    alpha: float = 2.0, want_wq: bool = False, want_loss: bool = False,
                    keep_factors: bool = False, sym: bool = False,
                    stream=None) -> QuantizedLinear:
    """GPTQ for one linear layer W (rows x n).  X: one calibration tensor
    (n x N) or an iterable of batches; or pass a ready Hessian H."""
    _need_cuda(W)
    rows, n = W.shape
    if H is None:
        if X is None:
            raise GptqError("give calibration inputs X or a Hessian H")
        H = torch.zeros(n, n, dtype=torch.float32, device=W.device)
        batches = [X] if isinstance(X, torch.Tensor) else X
        for xb in batches:
            gptq_hessian_accumulate(H, xb, alpha, stream=stream)
    cfg = make_config(bits, group_size, percdamp, actorder, sym=sym)
    U, perm, dead, info = gptq_cholesky_inverse(H, percdamp, actorder, stream=stream)
    q = gptq_quantize_layer(W, U, perm, dead, cfg, want_wq=want_wq, want_loss=want_loss,
                            stream=stream)
    if bits == 4 and n % 8 == 0:
        packed = gptq_pack_int4(q["codes"], stream=stream)
    elif bits == 3 and n % 32 == 0:
        packed = gptq_pack_int3(q["codes"], stream=stream)
    else:
        packed = q["codes"]
    return QuantizedLinear(packed, q["scales"], q["zeros"], q["g_idx"], perm, bits, group_size, n,
                           q["codes"], info, H if keep_factors else None,
                           U if keep_factors else None, q["Wq"], q["row_loss"])


class LayerQuantizer:
    """Repeated GPTQ of one layer shape with every buffer allocated once.

    ``run(W, X)`` enqueues the whole hot path on one stream, in order:
    H = 0, H += 2 X X^T, dead inputs / act-order / damping / U, the column
    sweep, packing, and dequantization to ``out_dtype``.  Outputs stay in the
    attributes (``H``, ``U``, ``perm``, ``dead``, ``info``, ``codes``,
    ``scales``, ``zeros``, ``g_idx``, ``packed``, ``deq`` and, if asked for,
    ``Wq`` and ``row_loss``).  ``events``: six CUDA events recorded around the
    five stages, for timing.  ``side``: the quantizer's own second stream,
    given to the factorisation and the sweep for their look-ahead
    (``lookahead=False``: everything on the caller's stream; same results).
    """

    STAGES = ("hessian", "cholesky_inverse", "sweep", "pack", "dequant")

    def __init__(self, rows: int, n: int, ntok: int, bits: int = 4, group_size: int = 128,
                 percdamp: float = 0.01, actorder: bool = False,
                 x_dtype: torch.dtype = torch.bfloat16, w_dtype: torch.dtype = torch.bfloat16,
                 out_dtype: torch.dtype = torch.bfloat16, want_wq: bool = False,
                 want_loss: bool = False, sym: bool = False, device=None,
                 lookahead: bool = True):
        if bits == 4 and n % 8:
            raise GptqError("int4 packing needs n % 8 == 0")
        if bits == 3 and n % 32:
            raise GptqError("int3 packing needs n % 32 == 0")
        if bits not in (3, 4):
            raise GptqError("packed storage is int3 or int4")
        dev = torch.device("cuda") if device is None else torch.device(device)
        self.rows, self.n, self.ntok, self.bits = rows, n, ntok, bits
        self.group_size, self.percdamp, self.actorder = group_size, percdamp, actorder
        self.cfg = make_config(bits, group_size, percdamp, actorder, sym=sym)
        G = 1 if group_size <= 0 else (n + group_size - 1) // group_size
        f32 = torch.float32
        self.H = torch.empty(n, n, dtype=f32, device=dev)
        self.U = torch.empty(n, n, dtype=f32, device=dev)
        self.perm = torch.empty(n, dtype=torch.int32, device=dev)
        self.dead = torch.empty(n, dtype=torch.uint8, device=dev)
        self.info = torch.zeros(1, dtype=torch.int32, device=dev)
        self.info_h = torch.zeros(1, dtype=torch.int32, device=dev)
        self.info_q = torch.zeros(1, dtype=torch.int32, device=dev)
        self.side = torch.cuda.Stream(dev) if lookahead else None
        self.codes = torch.empty(rows, n, dtype=torch.uint8, device=dev)
        self.scales = torch.empty(rows, G, dtype=f32, device=dev)
        self.zeros = torch.empty(rows, G, dtype=torch.uint8, device=dev)
        self.g_idx = torch.empty(n, dtype=torch.int32, device=dev)
        self.packed = torch.empty(rows, n * bits // 32, dtype=torch.int32, device=dev)
        self.deq = torch.empty(rows, n, dtype=out_dtype, device=dev)
        self.Wq = torch.empty(rows, n, dtype=f32, device=dev) if want_wq else None
        self.row_loss = torch.empty(rows, dtype=f32, device=dev) if want_loss else None
        self.ws_h = _workspace(gptq_workspace_size(GPTQ_OP_HESSIAN, 0, n, ntok, x_dtype), dev,
                               None)
        self.ws_c = _workspace(gptq_workspace_size(GPTQ_OP_CHOLESKY, 0, n), dev, None)
        self.ws_q = _workspace(gptq_workspace_size(GPTQ_OP_QUANTIZE, rows, n, 0, w_dtype,
                                                   self.cfg), dev, None)
        self._pack = gptq_pack_int4 if bits == 4 else gptq_pack_int3
        self.x_dtype, self.w_dtype = x_dtype, w_dtype
        self._stage = None        # run_streamed: two device staging buffers, device W, events

    def hessian(self, X: torch.Tensor, stream, mark=None) -> None:
        """H = 0, H += 2 X X^T on `stream`; mark(0) / mark(1) around the
        accumulation."""
        with torch.cuda.stream(stream):
            self.H.zero_()
        if mark:
            mark(0)
        gptq_hessian_accumulate(self.H, X, 2.0, ws=self.ws_h, info=self.info_h, stream=stream)
        if mark:
            mark(1)

    def finish(self, W: torch.Tensor, stream, mark=None) -> None:
        """Everything after the Hessian, on `stream`: U, the sweep, packing,
        dequantization.  mark(i) is called after stage i (2..5)."""
        gptq_cholesky_inverse(self.H, self.percdamp, self.actorder, self.U, self.perm, self.dead,
                              self.info, ws=self.ws_c, stream=stream, side_stream=self.side)
        if mark:
            mark(2)
        gptq_quantize_layer(W, self.U, self.perm, self.dead, self.cfg, self.codes, self.scales,
                            self.zeros, self.g_idx, self.Wq, self.row_loss, ws=self.ws_q,
                            info=self.info_q, stream=stream, side_stream=self.side)
        if mark:
            mark(3)
        self._pack(self.codes, self.packed, stream=stream)
        if mark:
            mark(4)
        gptq_dequant(self.packed, self.bits, self.n, self.scales, self.zeros, self.group_size,
                     self.g_idx, self.deq.dtype, out=self.deq, stream=stream)
        if mark:
            mark(5)

    def run_streamed(self, W_host: torch.Tensor, X_batches, stream=None):
        """The whole layer from inputs in (pinned) host memory: W and the
        calibration batches X_b (each n x N_b, contiguous) are copied in on a
        copy stream while H accumulates batch by batch on ``stream`` (page
        "GPTQ, with the code open", section "Paper vs. code": H is a sum over
        calibration batches), so the host-to-device copies overlap the
        Hessian.  Two device staging buffers of the largest batch take turns;
        a buffer is refilled only after the accumulation that read it.  The
        result equals ``run`` on the concatenated X up to the fp32 order of
        the Hessian's sums.

        Consecutive calls overlap: a call's copies wait only for the last
        reads of the buffers they overwrite (a staging buffer's previous
        accumulation, the device W's previous sweep), so they can run while
        the previous call's factorisation and sweep finish.  The host
        tensors must stay alive and unchanged until the copies are done (for
        example until ``stream`` has reached this call's end)."""
        s = torch.cuda.current_stream() if stream is None else stream
        dev = self.H.device
        if len(X_batches) == 0:
            raise GptqError("no calibration batch")
        for Xb in X_batches:
            if Xb.dim() != 2 or Xb.shape[0] != self.n or not Xb.is_contiguous() \
                    or Xb.dtype != self.x_dtype:
                raise GptqError("each batch must be a contiguous n x N_b tensor of the layer's "
                                "input dtype")
        if W_host.shape != (self.rows, self.n) or W_host.dtype != self.w_dtype:
            raise GptqError("W must be rows x n in the layer's weight dtype")
        nb = max(int(Xb.shape[1]) for Xb in X_batches)
        st = self._stage
        if st is None or st["cap"] < nb:
            st = {"cap": nb,
                  "buf": [torch.empty(self.n * nb, dtype=self.x_dtype, device=dev)
                          for _ in range(2)],
                  "W": torch.empty(self.rows, self.n, dtype=self.w_dtype, device=dev),
                  "copy": torch.cuda.Stream(dev),
                  "ev_w": torch.cuda.Event(), "ev_w_free": torch.cuda.Event(),
                  "ev_copied": [torch.cuda.Event(), torch.cuda.Event()],
                  "ev_used": [torch.cuda.Event(), torch.cuda.Event()]}
            if self._stage is not None:
                # new buffers: the old ones may still be read on s
                ev = torch.cuda.Event()
                ev.record(s)
                st["copy"].wait_event(ev)
            self._stage = st
        cs = st["copy"]
        # each staging buffer is overwritten once the accumulation that read
        # it last is done, W once the previous call's sweep has read it
        # (events never recorded yet make these waits no-ops).  W goes after
        # the first two batches, so that the copy stream does not hold those
        # behind the previous call's sweep.
        with torch.cuda.stream(s):
            self.H.zero_()
        w_after = min(1, len(X_batches) - 1)
        for i, Xb in enumerate(X_batches):
            slot = i % 2
            cs.wait_event(st["ev_used"][slot])
            dst = st["buf"][slot][: self.n * Xb.shape[1]].view(self.n, Xb.shape[1])
            with torch.cuda.stream(cs):
                dst.copy_(Xb, non_blocking=True)
            st["ev_copied"][slot].record(cs)
            if i == w_after:
                cs.wait_event(st["ev_w_free"])
                with torch.cuda.stream(cs):
                    st["W"].copy_(W_host, non_blocking=True)
                st["ev_w"].record(cs)
            s.wait_event(st["ev_copied"][slot])
            gptq_hessian_accumulate(self.H, dst, 2.0, ws=self.ws_h, info=self.info_h, stream=s)
            st["ev_used"][slot].record(s)
        s.wait_event(st["ev_w"])
        self.finish(st["W"], s)
        st["ev_w_free"].record(s)
        return self

    def run(self, W: torch.Tensor, X: torch.Tensor, stream=None, events=None):
        s = torch.cuda.current_stream() if stream is None else stream
        ev = events

        def mark(i):
            if ev is not None:
                ev[i].record(s)

        self.hessian(X, s, mark)
        self.finish(W, s, mark)
        return self

    def check_info(self) -> None:
        """Raises GptqError if a device status word reports a failure (syncs)."""
        ci, hi, qi = int(self.info.item()), int(self.info_h.item()), int(self.info_q.item())
        if ci != 0 or hi != 0 or qi != 0:
            raise GptqError(f"device status: cholesky info {ci}, hessian info {hi}, "
                            f"sweep info {qi}")


class LayerPipeline:
    """GPTQ of a sequence of linears, one layer at a time (page "GPTQ, with
    the code open", section "From one repair to a whole model": each layer is
    repaired from its own inputs and Hessian), with the Hessian of linear
    l + 1 accumulating on one stream while linear l is factored, swept,
    packed and dequantized on another.  The Hessian is tensor-core bound and
    the rest a chain of small dependent launches, so the two overlap on the
    SMs the chain leaves idle.

    ``shapes``: (rows, n) per linear; every linear sees ``ntok`` tokens.
    One LayerQuantizer per linear holds that linear's buffers and outputs
    (``layers[l]``).  ``run(Ws, Xs)`` enqueues everything and makes the
    caller's stream wait for the last linear.

    Measured on a 7B decoder block (7 linears, 65536 tokens each) the overlap
    gains nothing (0.96 to 1.00 of the one-stream time): the Hessian's
    persistent grid holds every SM, so the factorisation's and the sweep's
    kernels only get SMs when it ends.  So ``run`` uses the one-stream order
    unless ``overlap=True`` is asked for.
    """

    def __init__(self, shapes, ntok: int, bits: int = 4, group_size: int = 128,
                 percdamp: float = 0.01, actorder: bool = False, sym: bool = False,
                 x_dtype: torch.dtype = torch.bfloat16, w_dtype: torch.dtype = torch.bfloat16,
                 out_dtype: torch.dtype = torch.bfloat16, want_wq: bool = False,
                 want_loss: bool = False, device=None):
        dev = torch.device("cuda") if device is None else torch.device(device)
        self.layers = [LayerQuantizer(rows, n, ntok, bits, group_size, percdamp, actorder,
                                      x_dtype, w_dtype, out_dtype, want_wq, want_loss, sym=sym,
                                      device=dev)
                       for rows, n in shapes]
        self.s_h = torch.cuda.Stream(dev)
        self.s_q = torch.cuda.Stream(dev)
        self.ev_h = [torch.cuda.Event() for _ in shapes]
        self.ev_start = torch.cuda.Event()
        self.ev_done = torch.cuda.Event()

    def run(self, Ws, Xs, stream=None, overlap: bool = False):
        """overlap=False (the default) runs the work one linear after another
        on the caller's stream; overlap=True puts each next Hessian on a
        second stream (same results)."""
        s = torch.cuda.current_stream() if stream is None else stream
        if len(Ws) != len(self.layers) or len(Xs) != len(self.layers):
            raise GptqError("one W and one X per linear")
        if not overlap:
            for q, W, X in zip(self.layers, Ws, Xs):
                q.hessian(X, s)
                q.finish(W, s)
            return self
        self.ev_start.record(s)
        self.s_h.wait_event(self.ev_start)
        self.s_q.wait_event(self.ev_start)
        L = len(self.layers)
        for l in range(L + 1):
            if l < L:
                self.layers[l].hessian(Xs[l], self.s_h)
                self.ev_h[l].record(self.s_h)
            if l >= 1:
                self.s_q.wait_event(self.ev_h[l - 1])
                self.layers[l - 1].finish(Ws[l - 1], self.s_q)
        self.ev_done.record(self.s_q)
        s.wait_event(self.ev_done)
        return self

    def check_info(self) -> None:
        for q in self.layers:
            q.check_info()


# ----------------------------------------------------------------- low-rank adapters
def _on(idx: int, stream):
    """(context, stream handle) for a call on device idx: with a stream given,
    scratch and outputs allocated inside the context belong to that stream."""
    if stream is not None:
        if stream.device.index != idx:
            raise GptqError(f"the stream must be one of device {idx}, got {stream.device}")
        return torch.cuda.stream(stream), stream.cuda_stream
    if idx == _current_device():
        return _NO_CONTEXT, _raw_stream(idx)
    return torch.cuda.device(idx), _raw_stream(idx)


def _current_device() -> int:
    return torch.cuda.current_device()


def _raw_stream(idx: int) -> int:
    return torch.cuda.current_stream(idx).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):   # the same handles, without their wrappers
    _raw_stream = torch._C._cuda_getCurrentRawStream  # noqa: F811


_NO_CONTEXT = contextlib.nullcontext()


def _rows2d(t: torch.Tensor, name: str, rows: int, cols: int, device) -> int:
    """Row stride of a rows x cols tensor with contiguous rows on `device`."""
    if t.shape != (rows, cols):
        raise GptqError(f"{name} must be {rows} x {cols}, got {tuple(t.shape)}")
    if t.device != device:
        raise GptqError(f"{name} must live on {device}")
    ld, step = t.stride()
    if rows <= 1 and ld < cols:
        ld = cols
    if (step != 1 and cols > 1) or ld < cols:
        raise GptqError(f"{name} must have contiguous rows that do not overlap")
    return ld


class LowRankAdapters:
    """Low-rank adapters of one linear layer (rows x n), one per slot.

    A: (slots, max_rank, n), B: (slots, rows, max_rank), bf16 or fp32 (one
    type for both), each slot's rows contiguous.  ranks: int32 (slots,) or
    None (max_rank everywhere); scales: fp32 (slots,) or None (1).  The
    tensors stay the caller's: their values may change between calls (a
    training step, a slot loaded with another adapter), their storage must
    not: a call whose adapters have moved is refused.
    """

    def __init__(self, A: torch.Tensor, B: torch.Tensor, ranks: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None):
        _need_cuda(A, B, ranks, scales)
        if A.dim() != 3 or B.dim() != 3 or A.shape[0] != B.shape[0] or A.shape[1] != B.shape[2]:
            raise GptqError("A must be (slots, max_rank, n) and B (slots, rows, max_rank)")
        if A.dtype != B.dtype:
            raise GptqError("A and B must have the same dtype")
        wt = _dtype_code(A.dtype)
        for t in (B, ranks, scales):
            if t is not None and t.device != A.device:
                raise GptqError("adapters must live on one device")
        S, r, n = A.shape
        m = B.shape[1]
        strides = []
        for t, rows, cols in ((A, r, n), (B, m, r)):
            ld = cols if rows == 1 else t.stride(1)
            step = ld * rows if S <= 1 else t.stride(0)
            if (cols > 1 and t.stride(2) != 1) or ld < cols or step < ld * (rows - 1) + cols:
                raise GptqError("A and B must have contiguous rows that do not overlap")
            strides += [ld, step]
        for t, dt, name in ((ranks, torch.int32, "ranks"), (scales, torch.float32, "scales")):
            if t is not None and (t.dtype != dt or t.shape != (S,) or not t.is_contiguous()):
                raise GptqError(f"{name} must be a contiguous {dt} tensor of {S} slots")
        self.A, self.B, self.ranks, self.scales = A, B, ranks, scales
        self.slots, self.max_rank, self.n, self.rows = S, r, n, m
        self.device = A.device
        self._c = GptqLora(A.data_ptr(), B.data_ptr(), wt, S, r, n, m, strides[0], strides[1],
                           strides[2], strides[3], _p(ranks), _p(scales))
        self._ref = ctypes.byref(self._c)
        self._at = self._pointers()
        self._ws_size = {}
        self.workspace_size(0)     # checks the sizes

    def _pointers(self):
        return (self.A.data_ptr(), self.B.data_ptr(), _p(self.ranks), _p(self.scales))

    def workspace_size(self, ntok: int, backward: bool = False) -> int:
        """Bytes of scratch of gptq_lora_apply / gptq_lora_backward."""
        size = self._ws_size.get((ntok, backward))
        if size is None:
            out = ctypes.c_size_t(0)
            st = library().gptq_lora_workspace_size(self._ref, int(ntok), int(backward),
                                                    ctypes.byref(out))
            _check(st, "gptq_lora_workspace_size")
            if len(self._ws_size) > 256:     # a few token counts recur; any number may come
                self._ws_size.clear()
            size = self._ws_size[(ntok, backward)] = out.value
        return size


def _plan(ad: LowRankAdapters, plan, ntok: int):
    if ad._pointers() != ad._at:
        raise GptqError("the adapters' storage has moved: make a new LowRankAdapters")
    order, slot_start = plan
    i32, dev = torch.int32, ad.device
    if order.dtype != i32 or slot_start.dtype != i32 or order.shape != (ntok,) \
            or slot_start.shape != (ad.slots + 1,) or order.device != dev \
            or slot_start.device != dev or not order.is_contiguous() \
            or not slot_start.is_contiguous():
        raise GptqError(f"the plan must be contiguous int32 tensors of {ntok} tokens and "
                        f"{ad.slots} + 1 slots on {dev}")
    return order.data_ptr(), slot_start.data_ptr()


def gptq_lora_plan(ids: torch.Tensor, slots: int, order=None, slot_start=None, info=None,
                   stream=None):
    """The token plan (order, slot_start) of ids (int32, one slot per token,
    negative = no adapter); one plan serves every layer of a step.  info: a
    device int32 that becomes nonzero if an id was >= slots."""
    _need_cuda(ids, order, slot_start, info)
    if ids.dtype != torch.int32 or ids.dim() != 1 or not ids.is_contiguous():
        raise GptqError("ids must be a contiguous 1-D int32 tensor")
    ntok, slots = ids.shape[0], int(slots)
    for t, k in ((order, ntok), (slot_start, slots + 1), (info, 1)):
        if t is not None and (t.dtype != torch.int32 or t.numel() != k or not t.is_contiguous()
                              or t.device != ids.device):
            raise GptqError("order, slot_start and info must be contiguous int32 tensors of "
                            f"{ntok}, {slots + 1} and 1 elements on {ids.device}")
    ctx, s = _on(ids.device.index, stream)
    with ctx:
        if order is None:
            order = torch.empty(ntok, dtype=torch.int32, device=ids.device)
        if slot_start is None:
            slot_start = torch.empty(max(0, slots) + 1, dtype=torch.int32, device=ids.device)
        st = library().gptq_lora_plan(ids.data_ptr(), ntok, slots, order.data_ptr(),
                                      slot_start.data_ptr(), _p(info), s)
    _check(st, "gptq_lora_plan")
    return order, slot_start


def gptq_lora_apply(ad: LowRankAdapters, plan, x: torch.Tensor, y: torch.Tensor, u=None, ws=None,
                    stream=None) -> torch.Tensor:
    """y[t] += scale (x[t] A^T) B^T with each token's own adapter; returns y.
    x: (ntok, n), y: (ntok, rows), bf16 or fp32.  u: optional fp32 (ntok,
    max_rank) that receives x A^T for gptq_lora_backward."""
    ntok, dev = x.shape[0], ad.device
    ldx = _rows2d(x, "x", ntok, ad.n, dev)
    ldy = _rows2d(y, "y", ntok, ad.rows, dev)
    order, slot_start = _plan(ad, plan, ntok)
    ldu = 0
    if u is not None:
        if u.dtype != torch.float32:
            raise GptqError("u must be float32")
        ldu = _rows2d(u, "u", ntok, ad.max_rank, dev)
    ctx, s = _on(dev.index, stream)
    with ctx:
        wp = wn = 0
        need = ad.workspace_size(ntok) if u is None else 0
        if need:
            wp, wn = _aligned_ptr(_workspace(need, dev, ws))
        st = library().gptq_lora_apply(ad._ref, order, slot_start, ntok, x.data_ptr(),
                                       _dtype_code(x.dtype), ldx, y.data_ptr(),
                                       _dtype_code(y.dtype), ldy, _p(u), ldu, wp, wn, s)
    _check(st, "gptq_lora_apply")
    return y


def gptq_lora_backward(ad: LowRankAdapters, plan, dy: torch.Tensor, u=None, x=None, codes=None,
                       code_scales=None, group_size: int = 128, dx=None, dA=None, dB=None,
                       want_dA: bool = True, want_dB: bool = True, ws=None, stream=None):
    """Gradients of gptq_lora_apply: dx += (scale dy B) A in place (if given),
    dA (slots, max_rank, n) and dB (slots, rows, max_rank), fp32, written.
    The layer's input comes as x, or as 8-bit codes and code_scales of
    gptq_quantize_act8 with group_size.  Returns (dx, dA, dB)."""
    ntok, dev = dy.shape[0], ad.device
    lddy = _rows2d(dy, "dy", ntok, ad.rows, dev)
    order, slot_start = _plan(ad, plan, ntok)
    ldx = lddx = ldu = 0
    xt = GPTQ_F32
    if dA is not None or want_dA:
        if (x is None) == (codes is None):
            raise GptqError("give the layer's input as x or as codes")
        if x is not None:
            ldx, xt = _rows2d(x, "x", ntok, ad.n, dev), _dtype_code(x.dtype)
        else:
            if codes.dtype != torch.int8:
                raise GptqError("codes must be int8")
            ldx = _rows2d(codes, "codes", ntok, ad.n, dev)
            _check_act8_scales(code_scales, ntok, ad.n, group_size, dev)
    else:
        x = codes = None
    if dB is not None or want_dB:
        if u is None or u.dtype != torch.float32:
            raise GptqError("dB needs the float32 u of gptq_lora_apply")
        ldu = _rows2d(u, "u", ntok, ad.max_rank, dev)
    if dx is not None:
        lddx = _rows2d(dx, "dx", ntok, ad.n, dev)
    for t, shape, name in ((dA, (ad.slots, ad.max_rank, ad.n), "dA"),
                           (dB, (ad.slots, ad.rows, ad.max_rank), "dB")):
        if t is not None and (t.dtype != torch.float32 or t.shape != shape
                              or not t.is_contiguous() or t.device != dev):
            raise GptqError(f"{name} must be a contiguous float32 tensor {shape} on {dev}")
    ctx, s = _on(dev.index, stream)
    with ctx:
        if dA is None and want_dA:
            dA = torch.empty(ad.slots, ad.max_rank, ad.n, dtype=torch.float32, device=dev)
        if dB is None and want_dB:
            dB = torch.empty(ad.slots, ad.rows, ad.max_rank, dtype=torch.float32, device=dev)
        ws = _workspace(ad.workspace_size(ntok, True), dev, ws)
        wp, wn = _aligned_ptr(ws)
        st = library().gptq_lora_backward(
            ad._ref, order, slot_start, ntok, dy.data_ptr(), _dtype_code(dy.dtype), lddy, _p(x),
            xt, ldx, _p(codes), _p(code_scales) if codes is not None else None, int(group_size),
            _p(u) if dB is not None else None, ldu, _p(dx),
            GPTQ_F32 if dx is None else _dtype_code(dx.dtype), lddx, _p(dA), _p(dB), wp, wn, s)
    _check(st, "gptq_lora_backward")
    return dx, dA, dB


# ----------------------------------------------------------------- activations in 8 bits
def _act8_groups(n: int, group_size: int) -> int:
    if group_size not in (-1, 32, 64) and (group_size <= 0 or group_size % 128):
        raise GptqError(f"group_size must be -1, 32, 64 or a multiple of 128, got {group_size}")
    return 1 if group_size < 0 else (n + group_size - 1) // group_size


def _check_act8_scales(scales, rows: int, n: int, group_size: int, device) -> None:
    shape = (rows, _act8_groups(n, group_size))
    if scales is None or scales.dtype != torch.float32 or scales.shape != shape \
            or not scales.is_contiguous() or scales.device != device:
        raise GptqError(f"scales must be a contiguous float32 tensor {shape} on {device}")


def gptq_quantize_act8(x: torch.Tensor, group_size: int = 128, codes=None, scales=None,
                       stream=None):
    """(codes int8 (rows, n), scales fp32 (rows, G)) of x (rows x n, bf16 or
    fp32): scale = max |x| / 127 per row (group_size -1) or per group of 32,
    64 or a multiple of 128 columns, code = x / scale rounded half to even."""
    _need_cuda(x, codes, scales)
    if x.dim() != 2:
        raise GptqError("x must be a 2-D tensor")
    rows, n = x.shape
    dev = x.device
    ldx = _rows2d(x, "x", rows, n, dev)
    G = _act8_groups(n, group_size)
    ctx, s = _on(dev.index, stream)
    with ctx:
        if codes is None:
            codes = torch.empty(rows, n, dtype=torch.int8, device=dev)
        elif codes.dtype != torch.int8:
            raise GptqError("codes must be int8")
        if scales is None:
            scales = torch.empty(rows, G, dtype=torch.float32, device=dev)
        else:
            _check_act8_scales(scales, rows, n, group_size, dev)
        st = library().gptq_quantize_act8(x.data_ptr(), _dtype_code(x.dtype), rows, n, ldx,
                                          int(group_size), codes.data_ptr(),
                                          _rows2d(codes, "codes", rows, n, dev),
                                          scales.data_ptr(), s)
    _check(st, "gptq_quantize_act8")
    return codes, scales


def gptq_dequant_act8(codes: torch.Tensor, scales: torch.Tensor, group_size: int = 128, out=None,
                      out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """The values scale * code that gptq_quantize_act8's codes stand for."""
    _need_cuda(codes, scales, out)
    if codes.dim() != 2 or codes.dtype != torch.int8:
        raise GptqError("codes must be a 2-D int8 tensor")
    rows, n = codes.shape
    dev = codes.device
    ldc = _rows2d(codes, "codes", rows, n, dev)
    _check_act8_scales(scales, rows, n, group_size, dev)
    ctx, s = _on(dev.index, stream)
    with ctx:
        if out is None:
            out = torch.empty(rows, n, dtype=out_dtype, device=dev)
        st = library().gptq_dequant_act8(codes.data_ptr(), rows, n, ldc, scales.data_ptr(),
                                         int(group_size), out.data_ptr(), _dtype_code(out.dtype),
                                         _rows2d(out, "out", rows, n, dev), s)
    _check(st, "gptq_dequant_act8")
    return out


class AdaptedLinear:
    """A frozen quantized linear (a QuantizedLinear, or stored codes in the
    same layout) with low-rank adapters beside it.

    ``matvec`` serves: the packed codes are multiplied as they are
    (gptq_dequant_matvec) and the adapters' product is added, in fp32.
    ``forward`` and ``backward`` train the adapters: many tokens at once, so
    the weights are dequantized for one library product, and what is kept
    between the two is u (fp32, ntok x max_rank) and the input in 8 bits
    (``act_group``: the scales' group; None keeps the input itself).

    ``perm``: the codes are packed in sweep order (gptq_gather_columns_u8).
    """

    def __init__(self, packed, bits: int, n: int, scales, zeros, group_size: int,
                 adapters: LowRankAdapters, g_idx=None, perm=None, act_group: int | None = 128):
        if perm is not None and g_idx is not None:
            raise GptqError("perm (codes in sweep order) excludes g_idx")
        if bits not in (3, 4):
            raise GptqError("packed storage is int3 or int4")
        rows, dev = packed.shape[0], adapters.device
        if adapters.rows != rows or adapters.n != n:
            raise GptqError("the adapters must have the layer's rows and n")
        if n % (8 if bits == 4 else 32):
            raise GptqError("packed int4 needs n % 8 == 0, int3 n % 32 == 0")
        G = 1 if group_size <= 0 else (n + group_size - 1) // group_size
        if scales is None or scales.dim() != 2 or (g_idx is None and scales.shape[1] < G):
            raise GptqError(f"scales must be ({rows}, {G})")
        for t, dt, shape, name in ((packed, torch.int32, (rows, n * bits // 32), "packed"),
                                   (scales, torch.float32, (rows, scales.shape[1]), "scales"),
                                   (zeros, torch.uint8, scales.shape, "zeros"),
                                   (g_idx, torch.int32, (n,), "g_idx"),
                                   (perm, torch.int32, (n,), "perm")):
            if t is None and name in ("g_idx", "perm"):
                continue
            if t is None or t.dtype != dt or t.shape != shape or not t.is_contiguous() \
                    or t.device != dev:
                raise GptqError(f"{name} must be a contiguous {dt} tensor {tuple(shape)} on {dev}")
        if act_group is not None:
            _act8_groups(n, act_group)
        self.packed, self.bits, self.n, self.scales, self.zeros = packed, bits, n, scales, zeros
        self.group_size, self.g_idx, self.perm = group_size, g_idx, perm
        self.adapters, self.act_group = adapters, act_group
        self._place = None if perm is None else torch.argsort(perm.long())

    @classmethod
    def from_quantized(cls, q: QuantizedLinear, adapters: LowRankAdapters,
                       act_group: int | None = 128) -> "AdaptedLinear":
        return cls(q.packed, q.bits, q.n, q.scales, q.zeros, q.group_size, adapters,
                   g_idx=q.g_idx, act_group=act_group)

    def matvec(self, x: torch.Tensor, plan, stream=None) -> torch.Tensor:
        """y (ntok, rows) fp32 for x (ntok, n).  With a stream given, y and the
        scratch belong to that stream."""
        ad = self.adapters
        if x.dim() != 2:
            raise GptqError("x must be a 2-D tensor")
        _rows2d(x, "x", x.shape[0], ad.n, ad.device)
        _plan(ad, plan, x.shape[0])
        ctx, _ = _on(ad.device.index, stream)
        with ctx:
            y = gptq_dequant_matvec(self.packed, self.bits, self.n, self.scales, self.zeros, x,
                                    self.group_size, g_idx=self.g_idx, perm=self.perm,
                                    stream=stream)
            return gptq_lora_apply(ad, plan, x, y, stream=stream)

    def weight(self, dtype: torch.dtype) -> torch.Tensor:
        """The dequantized weights, columns in the layer's own order."""
        with _on(self.adapters.device.index, None)[0]:
            w = gptq_dequant(self.packed, self.bits, self.n, self.scales, self.zeros,
                             self.group_size, self.g_idx, dtype)
            return w if self._place is None else w[:, self._place]

    @torch.no_grad()
    def forward(self, x: torch.Tensor, plan):
        """(y, saved): y (ntok, rows) in x's dtype, saved for ``backward``.  y
        has no autograd graph: that would hold the base product alone."""
        y = torch.matmul(x, self.weight(x.dtype).t())
        u = torch.empty(x.shape[0], self.adapters.max_rank, dtype=torch.float32, device=x.device)
        gptq_lora_apply(self.adapters, plan, x, y, u=u)
        if self.act_group is None:
            return y, {"u": u, "x": x}
        codes, code_scales = gptq_quantize_act8(x, self.act_group)
        return y, {"u": u, "codes": codes, "code_scales": code_scales,
                   "group_size": self.act_group}

    @torch.no_grad()
    def backward(self, dy: torch.Tensor, plan, saved: dict):
        """(dx, dA, dB) from dy (ntok, rows): dx in dy's dtype, through the
        frozen weights and the adapters; dA and dB in fp32."""
        dx = torch.matmul(dy, self.weight(dy.dtype))
        return gptq_lora_backward(self.adapters, plan, dy, dx=dx, **saved)


# ----------------------------------------------------------------- checkpoint / resume
# Page "GPTQ, with the code open", section "From one repair to a whole model":
# a model is quantized one layer at a time, each from its own inputs.  For a
# long run over many linears, each finished linear's stored result is written
# to its own file, and a restarted run skips the linears whose files exist.

STORED_KEYS = ("packed", "scales", "zeros", "g_idx", "perm")


def save_quantized(path: str, outputs: dict, meta: dict) -> None:
    """Write one linear's stored result (host copies of ``STORED_KEYS`` and
    ``meta``) to ``path``.  The file appears only once it is complete: it is
    written under a temporary name and renamed, so an interrupted run leaves
    no partial result that a resumed run would take for a finished one."""
    import os
    blob = {k: outputs[k].detach().cpu() for k in STORED_KEYS if outputs.get(k) is not None}
    blob["meta"] = dict(meta)
    tmp = path + ".partial"
    torch.save(blob, tmp)
    os.replace(tmp, path)


def load_quantized(path: str) -> dict:
    return torch.load(path, map_location="cpu", weights_only=True)


def quantize_linears(names, quantize, out_dir: str, resume: bool = True) -> list:
    """Quantize the linears ``names`` in order with ``quantize(name) ->
    (outputs, meta)`` (``outputs`` holds at least ``packed``, ``scales`` and
    ``zeros`` of that linear), storing each under ``out_dir/<name>.pt``.  With
    ``resume``, a linear whose file already exists is not quantized again.
    Returns the names quantized by this call."""
    import os
    os.makedirs(out_dir, exist_ok=True)
    done = []
    for name in names:
        path = os.path.join(out_dir, f"{name}.pt")
        if resume and os.path.exists(path):
            continue
        outputs, meta = quantize(name)
        save_quantized(path, outputs, meta)
        done.append(name)
    return done


def layer_quantizer_outputs(lq: "LayerQuantizer") -> tuple:
    """(outputs, meta) of a LayerQuantizer after ``run``, for
    quantize_linears: checks ``info`` first (a failed linear is not stored)."""
    lq.check_info()
    outputs = {"packed": lq.packed, "scales": lq.scales, "zeros": lq.zeros,
               "g_idx": lq.g_idx if lq.actorder else None,
               "perm": lq.perm if lq.actorder else None}
    meta = {"rows": lq.rows, "n": lq.n, "bits": lq.bits, "group_size": lq.group_size,
            "actorder": bool(lq.actorder), "percdamp": lq.percdamp}
    return outputs, meta
