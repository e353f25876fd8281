"""Python binding of libflashsample (argument marshalling only).

Every step of sampling, of the 8-bit head and of beam search runs in the
library's HIP kernels; PyTorch supplies device memory and the current stream.
The function names follow the C ABI in include/flashsample.h and
include/flashsample_decode.h. Importing this module loads the library and fails
loudly if it has not been built (python -m lm_head_gemm_amd.build).
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch  # loads the HIP runtime the library binds to

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libflashsample.so")

FS_OK = 0
FS_ERR_INVALID_ARGUMENT = 1
FS_ERR_UNSUPPORTED = 2
FS_ERR_WORKSPACE_TOO_SMALL = 3
FS_ERR_HIP = 4

FS_DTYPE_BF16 = 0
FS_DTYPE_F32 = 1

FS_VARIANT_AUTO = 0
FS_VARIANT_GEMV = 1
FS_VARIANT_MFMA = 2

VARIANTS = {"auto": FS_VARIANT_AUTO, "gemv": FS_VARIANT_GEMV, "mfma": FS_VARIANT_MFMA}

FS_LAYOUT_ROWS = 0
FS_LAYOUT_TILED = 1


class FsOptions(ctypes.Structure):
    _fields_ = [
        ("variant", ctypes.c_int32),
        ("vocab_tile", ctypes.c_int32),
        ("logits", ctypes.c_void_p),
        ("ld_logits", ctypes.c_int64),
        ("logits_dtype", ctypes.c_int32),
        ("batch_tile", ctypes.c_int32),
        ("stage1_start", ctypes.c_void_p),
        ("stage1_stop", ctypes.c_void_p),
        ("weights_layout", ctypes.c_int32),
        ("single_pass", ctypes.c_int32),
        ("group_size", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


FS_BEAM_MAX = 64
FS_BEAM_MAX_STATES = 192


class FsBeamLayout(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int64) for name in
                ("outer", "outer_stride", "row_stride", "blocks", "block_stride", "block_bytes")]


class FlashSampleError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.fs_status_string(status).decode()
        if status == FS_ERR_HIP:
            msg += f" (hipError_t {_lib.fs_last_hip_error()})"
        super().__init__(f"{where}: {msg}")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m lm_head_gemm_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    c_i64, c_u64, c_sz, vp = ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t, ctypes.c_void_p
    lib.fs_status_string.restype = ctypes.c_char_p
    lib.fs_status_string.argtypes = [ctypes.c_int]
    lib.fs_last_hip_error.restype = ctypes.c_int
    lib.fs_num_vocab_tiles.restype = c_i64
    lib.fs_num_vocab_tiles.argtypes = [c_i64, c_i64, c_i64, ctypes.c_int, ctypes.POINTER(FsOptions)]
    lib.fs_vocab_tile_granule.restype = ctypes.c_int32
    lib.fs_vocab_tile_granule.argtypes = [ctypes.c_int]
    lib.fs_workspace_bytes.restype = c_sz
    lib.fs_workspace_bytes.argtypes = [c_i64, c_i64, c_i64, ctypes.c_int]
    lib.fs_workspace_bytes_ex.restype = c_sz
    lib.fs_workspace_bytes_ex.argtypes = [c_i64, c_i64, c_i64, ctypes.c_int, ctypes.POINTER(FsOptions)]
    fused = [vp, c_i64, vp, c_i64, ctypes.c_int, c_i64, c_i64, c_i64, ctypes.c_float, c_u64, c_u64,
             vp, c_sz, vp, vp]
    lib.fs_sample_fused.restype = ctypes.c_int
    lib.fs_sample_fused.argtypes = fused
    lib.fs_sample_fused_ex.restype = ctypes.c_int
    lib.fs_sample_fused_ex.argtypes = fused + [ctypes.POINTER(FsOptions)]
    lib.fs_sample_fused_noalloc.restype = ctypes.c_int
    lib.fs_sample_fused_noalloc.argtypes = [vp, c_i64, vp, c_i64, ctypes.c_int, c_i64, c_i64, c_i64,
                                            ctypes.c_float, c_u64, c_u64, vp, vp, ctypes.POINTER(FsOptions)]
    lib.fs_unfused_workspace_bytes.restype = c_sz
    lib.fs_unfused_workspace_bytes.argtypes = [c_i64, c_i64, c_i64, ctypes.c_int, ctypes.c_int]
    unfused = [vp, c_i64, vp, c_i64, ctypes.c_int, c_i64, c_i64, c_i64, ctypes.c_float, c_u64, c_u64,
               ctypes.c_int, vp, c_sz, vp, vp]
    lib.fs_sample_unfused.restype = ctypes.c_int
    lib.fs_sample_unfused.argtypes = unfused
    lib.fs_sample_unfused_ex.restype = ctypes.c_int
    lib.fs_sample_unfused_ex.argtypes = unfused + [ctypes.POINTER(FsOptions)]
    lib.fs_tiled_weights_bytes.restype = c_sz
    lib.fs_tiled_weights_bytes.argtypes = [c_i64, c_i64, ctypes.c_int]
    lib.fs_pack_weights_tiled.restype = ctypes.c_int
    lib.fs_pack_weights_tiled.argtypes = [vp, c_i64, c_i64, c_i64, ctypes.c_int, vp, c_sz, vp]
    lib.fs_test_philox.restype = ctypes.c_int
    lib.fs_test_philox.argtypes = [c_u64, c_u64, c_i64, c_i64, c_i64, vp, vp]
    lib.fs_test_gumbel.restype = ctypes.c_int
    lib.fs_test_gumbel.argtypes = [vp, c_i64, vp, vp]
    lib.fs_workspace_reset.restype = ctypes.c_int
    lib.fs_workspace_reset.argtypes = [vp, c_sz, vp]
    lib.fs_probe_read_blocks.restype = c_i64
    lib.fs_probe_read_blocks.argtypes = [c_i64, c_i64]
    lib.fs_probe_read.restype = ctypes.c_int
    lib.fs_probe_read.argtypes = [vp, c_i64, c_i64, vp, vp]
    lib.fs_quantize_i8.restype = ctypes.c_int
    lib.fs_quantize_i8.argtypes = [vp, c_i64, ctypes.c_int, c_i64, c_i64, vp, c_i64, vp, vp]
    lib.fs_rms_norm_i8.restype = ctypes.c_int
    lib.fs_rms_norm_i8.argtypes = [vp, c_i64, vp, c_i64, vp, ctypes.c_int, ctypes.c_int, c_i64, c_i64,
                                   ctypes.c_float, vp, c_i64, vp, c_i64, vp, vp]
    product = [vp, c_i64, vp, vp, c_i64, vp, c_i64, c_i64, c_i64]
    lib.fs_matmul_i8.restype = ctypes.c_int
    lib.fs_matmul_i8.argtypes = product + [vp, c_i64, ctypes.c_int, vp]
    lib.fs_sample_i8_workspace_bytes.restype = c_sz
    lib.fs_sample_i8_workspace_bytes.argtypes = [c_i64, c_i64, c_i64]
    lib.fs_sample_i8.restype = ctypes.c_int
    lib.fs_sample_i8.argtypes = product + [ctypes.c_float, c_u64, c_u64, vp, c_sz, vp, vp]
    lib.fs_beam_select_workspace_bytes.restype = c_sz
    lib.fs_beam_select_workspace_bytes.argtypes = [c_i64, c_i64, c_i64, c_i64, ctypes.c_int]
    lib.fs_beam_select.restype = ctypes.c_int
    lib.fs_beam_select.argtypes = [vp, c_i64, ctypes.c_int, vp, vp, ctypes.c_int32, c_i64, c_i64, c_i64, c_i64,
                                   vp, c_sz, vp, vp, vp, vp]
    layout = ctypes.POINTER(FsBeamLayout)
    lib.fs_beam_reorder.restype = ctypes.c_int
    lib.fs_beam_reorder.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), c_i64, layout, layout, vp, c_i64,
                                    c_i64, vp]
    return lib


_lib = _load()


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return FS_DTYPE_BF16
    if t == torch.float32:
        return FS_DTYPE_F32
    raise TypeError(f"unsupported dtype {t}")


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


# The current stream's handle of a device, without the Python object around it
# (2.7 us per call); torch builds without the function take the long way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _check(st: int, where: str):
    if st != FS_OK:
        raise FlashSampleError(st, where)


class TiledWeights:
    """A bf16 LM head [V, D] repacked once into the tiled layout
    (fs_pack_weights_tiled): blocks of 16 vocab rows x 256 columns, each 8 KiB
    contiguous in matrix-core operand order. Pass it wherever W is taken."""

    def __init__(self, W: torch.Tensor, stream=None):
        if not W.is_cuda or W.dtype != torch.bfloat16 or W.dim() != 2 or W.stride(1) != 1:
            raise ValueError("TiledWeights needs a bf16 device tensor [V, D] with contiguous rows")
        self.V, self.D = W.shape
        nbytes = int(_lib.fs_tiled_weights_bytes(self.V, self.D, FS_DTYPE_BF16))
        self.data = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
        _check(_lib.fs_pack_weights_tiled(W.data_ptr(), W.stride(0), self.V, self.D, FS_DTYPE_BF16,
                                          self.data.data_ptr(), nbytes, _stream(stream)),
               "fs_pack_weights_tiled")
        self.dtype = W.dtype
        self.device = W.device

    @property
    def shape(self):
        return (self.V, self.D)


def _weights(W):
    """(pointer, ldw, V, D, layout) of a row-major tensor or TiledWeights."""
    if isinstance(W, TiledWeights):
        return W.data.data_ptr(), W.D, W.V, W.D, FS_LAYOUT_TILED
    return W.data_ptr(), W.stride(0), W.shape[0], W.shape[1], FS_LAYOUT_ROWS


def _check_inputs(H: torch.Tensor, W):
    if not (H.is_cuda and W.device.type == "cuda"):
        raise ValueError("H and W must be device tensors")
    if H.dim() != 2 or len(W.shape) != 2 or H.shape[1] != W.shape[1]:
        raise ValueError(f"H [B, D] and W [V, D] expected, got {tuple(H.shape)} and {tuple(W.shape)}")
    if H.dtype != W.dtype:
        raise ValueError("H and W must share a dtype")
    if H.stride(1) != 1 or (isinstance(W, torch.Tensor) and W.stride(1) != 1):
        raise ValueError("H and W rows must be contiguous")


def make_options(variant="auto", vocab_tile=0, logits=None, events=None, batch_tile=0,
                 layout=FS_LAYOUT_ROWS, single_pass=False, group_size=0) -> FsOptions:
    o = FsOptions()
    o.single_pass = int(bool(single_pass))
    o.group_size = int(group_size)
    o.variant = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    o.vocab_tile = int(vocab_tile)
    o.batch_tile = int(batch_tile)
    o.weights_layout = int(layout)
    if logits is not None:
        o.logits = logits.data_ptr()
        o.ld_logits = logits.stride(0)
        o.logits_dtype = _dtype_code(logits.dtype)
    if events is not None:
        o.stage1_start = events[0].cuda_event
        o.stage1_stop = events[1].cuda_event
    return o


def workspace_reset(workspace: torch.Tensor, stream=None) -> None:
    """Zeroes a workspace with the library's fill kernel (fs_workspace_reset)."""
    _check(_lib.fs_workspace_reset(workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                   _stream(stream)), "fs_workspace_reset")


def num_vocab_tiles(B, D, V, dtype=torch.bfloat16, variant="auto", vocab_tile=0, tiled=False) -> int:
    o = make_options(variant, vocab_tile, layout=FS_LAYOUT_TILED if tiled else FS_LAYOUT_ROWS)
    return int(_lib.fs_num_vocab_tiles(B, D, V, _dtype_code(dtype), ctypes.byref(o)))


def workspace_bytes(B, D, V, dtype=torch.bfloat16, variant="auto", vocab_tile=0, tiled=False,
                    single_pass=False, group_size=0, batch_tile=0) -> int:
    o = make_options(variant, vocab_tile, layout=FS_LAYOUT_TILED if tiled else FS_LAYOUT_ROWS,
                     single_pass=single_pass, group_size=group_size, batch_tile=batch_tile)
    return int(_lib.fs_workspace_bytes_ex(B, D, V, _dtype_code(dtype), ctypes.byref(o)))


def unfused_workspace_bytes(B, D, V, dtype=torch.bfloat16, logits_dtype=torch.bfloat16) -> int:
    return int(_lib.fs_unfused_workspace_bytes(B, D, V, _dtype_code(dtype), _dtype_code(logits_dtype)))


def sample_fused(H: torch.Tensor, W, temperature: float, seed: int, step: int,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 variant="auto", vocab_tile: int = 0, logits: torch.Tensor | None = None,
                 events=None, stream=None, batch_tile: int = 0, single_pass: bool = False,
                 group_size: int = 0) -> torch.Tensor:
    """One token per row of H from softmax(H W^T / T) (Gumbel-max, fused).
    W is a row-major [V, D] tensor or a TiledWeights. With single_pass, a
    caller-provided workspace must have been zeroed once (workspace_reset).
    group_size > 0 selects the grouped variant (bf16; tiled weights, or
    row-major ones with D a multiple of 256): the group of group_size vocab
    entries is drawn from its log-mass, the token is that group's local
    Gumbel-max sample."""
    _check_inputs(H, W)
    B, D = H.shape
    wptr, ldw, V, _, layout = _weights(W)
    o = make_options(variant, vocab_tile, logits, events, batch_tile, layout, single_pass, group_size)
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=H.device)
    if workspace is None:
        nbytes = int(_lib.fs_workspace_bytes_ex(B, D, V, _dtype_code(H.dtype), ctypes.byref(o)))
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=H.device)
        if single_pass:
            workspace_reset(workspace, stream)
    st = _lib.fs_sample_fused_ex(H.data_ptr(), H.stride(0), wptr, ldw, _dtype_code(H.dtype), B, D, V,
                                 float(temperature), int(seed), int(step), workspace.data_ptr(),
                                 workspace.numel(), out.data_ptr(), _stream(stream), ctypes.byref(o))
    _check(st, "fs_sample_fused_ex")
    return out


# Bytes of the library's static per-GPU scratch array (FS_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 8 << 20


def sample_fused_noalloc(H: torch.Tensor, W, temperature: float, seed: int, step: int,
                         out: torch.Tensor | None = None, variant="auto", vocab_tile: int = 0,
                         logits: torch.Tensor | None = None, stream=None, batch_tile: int = 0,
                         single_pass: bool = False, group_size: int = 0) -> torch.Tensor:
    """sample_fused without a workspace (fs_sample_fused_noalloc): the library
    uses its static per-GPU scratch array instead, so the C call allocates
    nothing. Calls on one GPU must not overlap in time."""
    _check_inputs(H, W)
    B, D = H.shape
    wptr, ldw, V, _, layout = _weights(W)
    o = make_options(variant, vocab_tile, logits, None, batch_tile, layout, single_pass, group_size)
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=H.device)
    st = _lib.fs_sample_fused_noalloc(H.data_ptr(), H.stride(0), wptr, ldw, _dtype_code(H.dtype), B, D, V,
                                      float(temperature), int(seed), int(step), out.data_ptr(), _stream(stream),
                                      ctypes.byref(o))
    _check(st, "fs_sample_fused_noalloc")
    return out


def sample_unfused(H: torch.Tensor, W, temperature: float, seed: int, step: int,
                   logits_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None, variant="auto",
                   vocab_tile: int = 0, batch_tile: int = 0) -> torch.Tensor:
    """The IO-model baseline: GEMM writes logits, a sampler kernel reads them."""
    _check_inputs(H, W)
    B, D = H.shape
    wptr, ldw, V, _, layout = _weights(W)
    o = make_options(variant, vocab_tile, None, None, batch_tile, layout)
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=H.device)
    if workspace is None:
        nbytes = unfused_workspace_bytes(B, D, V, H.dtype, logits_dtype)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=H.device)
    st = _lib.fs_sample_unfused_ex(H.data_ptr(), H.stride(0), wptr, ldw, _dtype_code(H.dtype), B, D, V,
                                   float(temperature), int(seed), int(step), _dtype_code(logits_dtype),
                                   workspace.data_ptr(), workspace.numel(), out.data_ptr(), _stream(stream),
                                   ctypes.byref(o))
    _check(st, "fs_sample_unfused_ex")
    return out


def test_philox(seed: int, step: int, b: int, v0: int, n: int, device="cuda") -> torch.Tensor:
    out = torch.empty(n, dtype=torch.int32, device=device)
    _check(_lib.fs_test_philox(seed, step, b, v0, n, out.data_ptr(), _stream(None)), "fs_test_philox")
    return out


def test_gumbel(words: torch.Tensor) -> torch.Tensor:
    assert words.dtype == torch.int32 and words.is_cuda and words.is_contiguous()
    out = torch.empty(words.numel(), dtype=torch.float32, device=words.device)
    _check(_lib.fs_test_gumbel(words.data_ptr(), words.numel(), out.data_ptr(), _stream(None)),
           "fs_test_gumbel")
    return out


def probe_read(src: torch.Tensor, chunk_bytes: int = 1 << 19, sink: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Streams all bytes of a contiguous device tensor (see fs_probe_read)."""
    assert src.is_cuda and src.is_contiguous()
    nbytes = src.numel() * src.element_size()
    nblk = int(_lib.fs_probe_read_blocks(nbytes, chunk_bytes))
    if nblk < 0:
        raise ValueError("probe_read: bytes and chunk must be positive multiples of 16")
    if sink is None:
        sink = torch.empty(nblk, dtype=torch.int32, device=src.device)
    _check(_lib.fs_probe_read(src.data_ptr(), nbytes, chunk_bytes, sink.data_ptr(), _stream(stream)),
           "fs_probe_read")
    return sink


# ------------------------------------------------------- 8-bit head, beam search
_NOWHERE_ELSE = contextlib.nullcontext()


def _on(device: torch.device, stream):
    """Where a call on tensors of `device` allocates and launches: on `stream`
    (a torch stream of that device), or on that device's current stream. What
    is allocated within belongs to that stream, so its memory is not handed on
    while the call still runs there."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream)
    if device.index != _current_device():
        return torch.cuda.device(device)
    return _NOWHERE_ELSE


def _same_device(x: torch.Tensor, *others) -> torch.device:
    at = x.get_device()
    if at < 0:
        raise ValueError("device tensors expected")
    for t in others:
        if t is not None and t.get_device() != at:
            raise ValueError(f"tensors on one device expected, got {x.device} and {t.device}")
    return x.device


def _expect(t: torch.Tensor, shape, dtype, what: str):
    """A contiguous tensor of this shape and dtype."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{what}: {dtype} {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: contiguous elements expected")


def _rows(t: torch.Tensor, shape, dtype, what: str) -> int:
    """A 2-D tensor of this shape and dtype with contiguous rows; its row stride
    (torch leaves the stride of a single row open)."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{what}: {dtype} {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")
    if t.is_contiguous():
        return shape[1]
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{what}: contiguous rows expected")
    return ld if shape[0] > 1 else max(ld, shape[1])


def _matrix(t: torch.Tensor, what: str):
    if t.dim() != 2:
        raise ValueError(f"{what}: [rows, columns] expected, got {tuple(t.shape)}")
    return tuple(t.shape)


def _workspace(t: torch.Tensor) -> int:
    """Bytes of a given workspace."""
    if not t.is_contiguous():
        raise ValueError("workspace: contiguous elements expected")
    return t.numel() * t.element_size()


def _codes(x, shape, q, scales):
    """Codes and scales for rows like x's, made where not given, and the codes' row stride."""
    if q is None:
        q, ldq = x.new_empty(*shape, dtype=torch.int8), shape[1]
    else:
        ldq = _rows(q, shape, torch.int8, "q")
    if scales is None:
        scales = x.new_empty(shape[0], dtype=torch.float32)
    else:
        _expect(scales, shape[:1], torch.float32, "scales")
    return q, ldq, scales


def quantize_i8(x: torch.Tensor, q: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """Rows of x [M, D] (bf16 or fp32) as 8-bit codes and one scale per row:
    (q int8 [M, D], scales fp32 [M]) with x ~ q * scales[:, None]
    (fs_quantize_i8). Brings an LM head [V, D] to 8 bits (once, when it is
    loaded) and hidden states that are normed already."""
    shape = _matrix(x, "x")
    dt, ldx = _dtype_code(x.dtype), _rows(x, shape, x.dtype, "x")
    device = _same_device(x, q, scales)
    with _on(device, stream):
        q, ldq, scales = _codes(x, shape, q, scales)
        st = _lib.fs_quantize_i8(x.data_ptr(), ldx, dt, *shape, q.data_ptr(), ldq, scales.data_ptr(),
                                 _raw_stream(device.index))
    _check(st, "fs_quantize_i8")
    return q, scales


def rms_norm_i8(x: torch.Tensor, gain: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                sum_out: torch.Tensor | None = None, q: torch.Tensor | None = None,
                scales: torch.Tensor | None = None, stream=None):
    """Root-mean-square norm of x (+ residual), times gain [D], as 8-bit codes
    and one scale per row (fs_rms_norm_i8): (q, scales), and with a residual
    (q, scales, h), h = x + residual in x's dtype. h goes to sum_out if given,
    which may be x or residual itself. gain is in x's dtype or fp32."""
    shape = _matrix(x, "x")
    dt, ldx = _dtype_code(x.dtype), _rows(x, shape, x.dtype, "x")
    _expect(gain, shape[1:], gain.dtype, "gain")
    gt = _dtype_code(gain.dtype)
    res = ldr = into = ldi = 0
    if residual is not None:
        res, ldr = residual.data_ptr(), _rows(residual, shape, x.dtype, "residual")
    elif sum_out is not None:
        raise ValueError("sum_out without a residual")
    device = _same_device(x, gain, residual, sum_out, q, scales)
    with _on(device, stream):
        if residual is not None:
            if sum_out is None:
                sum_out = x.new_empty(*shape)
            into, ldi = sum_out.data_ptr(), _rows(sum_out, shape, x.dtype, "sum_out")
        q, ldq, scales = _codes(x, shape, q, scales)
        st = _lib.fs_rms_norm_i8(x.data_ptr(), ldx, res, ldr, gain.data_ptr(), gt, dt, *shape, eps, into, ldi,
                                 q.data_ptr(), ldq, scales.data_ptr(), _raw_stream(device.index))
    _check(st, "fs_rms_norm_i8")
    return (q, scales) if residual is None else (q, scales, sum_out)


def _product_inputs(q, q_scales, w, w_scales):
    """(M, N, K) and the row strides of checked operands."""
    (M, K), (N, _) = _matrix(q, "q"), _matrix(w, "w")
    ldq, ldw = _rows(q, (M, K), torch.int8, "q"), _rows(w, (N, K), torch.int8, "w")
    _expect(q_scales, (M,), torch.float32, "q_scales")
    _expect(w_scales, (N,), torch.float32, "w_scales")
    return M, N, K, ldq, ldw


def matmul_i8(q: torch.Tensor, q_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
              out: torch.Tensor | None = None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """(q * q_scales[:, None]) @ (w * w_scales[:, None]).T of 8-bit codes q
    [M, K] and w [N, K], summed exactly in integers (fs_matmul_i8): [M, N] in
    out's dtype, or out_dtype (bf16 or fp32). K is a multiple of 16."""
    M, N, K, ldq, ldw = _product_inputs(q, q_scales, w, w_scales)
    device = _same_device(q, q_scales, w, w_scales, out)
    with _on(device, stream):
        if out is None:
            dt, ldo = _dtype_code(out_dtype), N
            out = q.new_empty(M, N, dtype=out_dtype)
        else:
            dt, ldo = _dtype_code(out.dtype), _rows(out, (M, N), out.dtype, "out")
        st = _lib.fs_matmul_i8(q.data_ptr(), ldq, q_scales.data_ptr(), w.data_ptr(), ldw, w_scales.data_ptr(),
                               M, N, K, out.data_ptr(), ldo, dt, _raw_stream(device.index))
    _check(st, "fs_matmul_i8")
    return out


def sample_i8_workspace_bytes(B, D, V) -> int:
    return int(_lib.fs_sample_i8_workspace_bytes(B, D, V))


def sample_i8(q: torch.Tensor, q_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, temperature: float,
              seed: int, step: int, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """One token per row from softmax(l / T), l = matmul_i8's fp32 logits of
    codes q [B, D] and an 8-bit LM head w [V, D] (fs_sample_i8). Noise, ties
    and NaN rule are sample_fused's."""
    B, V, D, ldq, ldw = _product_inputs(q, q_scales, w, w_scales)
    device = _same_device(q, q_scales, w, w_scales, out, workspace)
    with _on(device, stream):
        if out is None:
            out = torch.empty(B, dtype=torch.int32, device=q.device)
        else:
            _expect(out, (B,), torch.int32, "out")
        if workspace is None:
            workspace = torch.empty(max(sample_i8_workspace_bytes(B, D, V), 256), dtype=torch.uint8, device=q.device)
        st = _lib.fs_sample_i8(q.data_ptr(), ldq, q_scales.data_ptr(), w.data_ptr(), ldw, w_scales.data_ptr(),
                               B, D, V, float(temperature), int(seed), int(step), workspace.data_ptr(),
                               _workspace(workspace), out.data_ptr(), _raw_stream(device.index))
    _check(st, "fs_sample_i8")
    return out


@functools.lru_cache(maxsize=64)   # by sizes only
def _select_bytes(B, beams, V, n, dt) -> int:
    return max(int(_lib.fs_beam_select_workspace_bytes(B, beams, V, n, dt)), 256)


def beam_select_workspace_bytes(B, beams, V, n, dtype=torch.bfloat16) -> int:
    return int(_lib.fs_beam_select_workspace_bytes(B, beams, V, n, _dtype_code(dtype)))


def beam_select(logits: torch.Tensor, scores: torch.Tensor, n: int | None = None,
                finished: torch.Tensor | None = None, pad_token: int = 0, out=None,
                workspace: torch.Tensor | None = None, stream=None):
    """The n best continuations (default: as many as beams) of each group of
    beams, from logits [B * beams, V] (bf16 or fp32) and scores fp32
    [B, beams]: (scores fp32, parents int32, tokens int32), each [B, n], best
    first (fs_beam_select). A beam marked in finished (bool or uint8
    [B, beams]) stands for itself once, with pad_token. out: the three output
    tensors; the scores may go to `scores` itself where n is beams."""
    B, beams = _matrix(scores, "scores")
    _expect(scores, (B, beams), torch.float32, "scores")
    R, V = shape = _matrix(logits, "logits")
    if R != B * beams:
        raise ValueError(f"logits: {B * beams} rows expected, got {R}")
    dt, ld = _dtype_code(logits.dtype), _rows(logits, shape, logits.dtype, "logits")
    n = beams if n is None else int(n)
    if not -2**31 <= pad_token < 2**31:
        raise ValueError(f"pad_token {pad_token} is no token")
    done = 0
    if finished is not None:
        if finished.dtype not in (torch.bool, torch.uint8):
            raise ValueError(f"finished: bool or uint8 expected, got {finished.dtype}")
        _expect(finished, (B, beams), finished.dtype, "finished")
        done = finished.data_ptr()
    given = out if out is not None else ()
    device = _same_device(logits, scores, finished, workspace, *given)
    with _on(device, stream):
        if out is None:
            out = (logits.new_empty(B, n, dtype=torch.float32), logits.new_empty(B, n, dtype=torch.int32),
                   logits.new_empty(B, n, dtype=torch.int32))
        else:
            for t, dtype, what in zip(out, (torch.float32, torch.int32, torch.int32),
                                      ("out scores", "out parents", "out tokens"), strict=True):
                _expect(t, (B, n), dtype, what)
        if workspace is None:
            workspace = logits.new_empty(_select_bytes(B, beams, V, n, dt), dtype=torch.uint8)
        st = _lib.fs_beam_select(logits.data_ptr(), ld, dt, scores.data_ptr(), done, int(pad_token), B, beams, V, n,
                                 workspace.data_ptr(), _workspace(workspace),
                                 out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), _raw_stream(device.index))
    _check(st, "fs_beam_select")
    return tuple(out)


def _fold(dims):
    """Dimensions (size, strides in bytes of each tensor) from the outermost
    in, joined where the next one continues the one before in every tensor,
    those of size 1 left out."""
    folded = []
    for size, strides in dims:
        if size == 1:
            continue
        if folded and folded[-1][1] == tuple(size * s for s in strides):
            folded[-1] = (folded[-1][0] * size, strides)
        else:
            folded.append((size, strides))
    return folded


def _beam_layouts(dim: int, *tensors: torch.Tensor):
    """For each of some state tensors of one shape and dtype, whose rows are
    dimension dim: its FsBeamLayout, alike but for the strides, and the byte
    offsets of the slabs that a layout does not reach."""
    return _layouts(dim, tensors[0].element_size(), tensors[0].shape, *(t.stride() for t in tensors))


@functools.lru_cache(maxsize=64)   # shapes and strides of a decode loop come again
def _layouts(dim, e, shape, *tensors):
    dims = [(n, tuple(s * e for s in strides)) for n, strides in zip(shape, zip(*tensors))]
    one, none = (1,) * len(tensors), (0,) * len(tensors)
    outer, inner = _fold(dims[:dim]), _fold(dims[dim + 1:] + [(e, one)])
    block = inner.pop()[0] if inner and inner[-1][1] == one else 1
    if len(inner) > 1:
        raise ValueError("beam_reorder: strides " + ", ".join(map(str, tensors)) +
                         f" of {tuple(shape)} leave more than one run of blocks")
    blocks = inner[0] if inner else (1, none)
    slab = outer.pop() if outer else (1, none)
    layouts = []
    for i in range(len(tensors)):
        starts = [0]
        for n, s in outer:
            starts = [o + k * s[i] for o in starts for k in range(n)]
        layouts.append((FsBeamLayout(slab[0], slab[1][i], dims[dim][1][i], blocks[0], blocks[1][i], block), starts))
    return layouts


def beam_reorder(states, parents: torch.Tensor, dim: int = 0, out=None, stream=None):
    """Row b * beams + i of every state becomes the former row
    b * beams + parents[b, i] (fs_beam_reorder). states: a tensor, or a list
    of tensors of one shape, strides and dtype (say each layer's keys and
    values), with B * beams rows in dimension dim; views are welcome, so a
    cache is passed as far as it is filled (cache[:, :, :length]). parents:
    int32 [B, beams]; a row whose parent is not in 0 .. beams - 1 stays as it
    is. out: None (in place), or like states. Returns what was written."""
    tensors = [states] if isinstance(states, torch.Tensor) else list(states)
    targets = tensors if out is None else [out] if isinstance(out, torch.Tensor) else list(out)
    B, beams = _matrix(parents, "parents")
    _expect(parents, (B, beams), torch.int32, "parents")
    if not tensors:
        raise ValueError("no states")
    if len(targets) != len(tensors):
        raise ValueError(f"{len(tensors)} states and {len(targets)} outputs")
    first = tensors[0]
    dim = dim + first.dim() if dim < 0 else dim
    if not 0 <= dim < first.dim() or first.shape[dim] != B * beams:
        raise ValueError(f"states with {B * beams} rows in dimension {dim} expected, got {tuple(first.shape)}")
    for group, like in ((tensors, first), (targets, targets[0])):
        for t in group:
            if t.shape != first.shape or t.dtype != first.dtype or t.stride() != like.stride():
                raise ValueError("states (and outputs) of one shape, strides and dtype expected")
    device = _same_device(first, parents, *tensors, *targets)
    written = states if out is None else out
    if first.numel() == 0:
        return written
    if targets is tensors or all(t.data_ptr() == u.data_ptr() and t.stride() == u.stride()
                                 for t, u in zip(tensors, targets)):
        (layout, starts), = _beam_layouts(dim, first)
        to, dst = layout, None
    else:
        (layout, starts), (to, to_starts) = _beam_layouts(dim, first, targets[0])
        dst = [t.data_ptr() + s for t in targets for s in to_starts]
    src = [t.data_ptr() + s for t in tensors for s in starts]
    if len(src) > FS_BEAM_MAX_STATES:
        raise ValueError(f"beam_reorder: more than {FS_BEAM_MAX_STATES} separate buffers in one call")
    table = ctypes.c_void_p * len(src)
    with _on(device, stream):
        st = _lib.fs_beam_reorder(table(*src), None if dst is None else table(*dst), len(src), ctypes.byref(layout),
                                  None if dst is None else ctypes.byref(to), parents.data_ptr(), B, beams,
                                  _raw_stream(device.index))
    _check(st, "fs_beam_reorder")
    return written
