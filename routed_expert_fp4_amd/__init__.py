"""Python binding of libroutedfp4 (the MI355X routed-expert FFN library).

Argument marshalling only: every step of the layer runs in the HIP kernels behind
the C ABI declared in ``include/routed_fp4.h``.  The functions carry the C names;
they take torch tensors that already live on the GPU, check dtype, shape, device
and contiguity, pass raw pointers and the current HIP stream, and raise
``MoeError`` on any non-OK status.  PyTorch is used for device memory and
streams only.

If the shared library has not been built this module raises on first use; there
is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libroutedfp4.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_DEVICE = 0, -1, -2, -3, -4
MOE_FMT_MXFP4, MOE_FMT_NVFP4 = 1, 2
MOE_NUM_TENSORS = 7
MOE_MAX_EXPERTS, MOE_MAX_TOPK, MOE_MAX_DECODE_TOKENS, MOE_MAX_TOKENS = 1024, 32, 16, 4096
BLOCK = {MOE_FMT_MXFP4: 32, MOE_FMT_NVFP4: 16}

EXPORTS = ("moe_version", "moe_status_string", "moe_bank_layout", "moe_workspace_size",
           "moe_workspace_init", "moe_route", "moe_expert_fwd", "moe_layer_fwd", "moe_dequant",
           "moe_latent_workspace_size", "moe_latent_layer_fwd", "moe_mx_mma_workspace_size",
           "moe_expert_fwd_mx_mma", "moe_layer_fwd_noalloc", "moe_quant_workspace_size",
           "moe_quant_linear", "moe_expert_counts", "moe_balance_workspace_size",
           "moe_balance_fwd", "moe_balance_bwd", "moe_route_bwd")
MOE_DT_F32, MOE_DT_BF16, MOE_DT_F16 = 1, 2, 3
MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX = 1, 2
MOE_MAX_QUANT_ROWS, MOE_MAX_QUANT_COLS = 1 << 22, 1 << 17
MOE_MAX_BATCH_TOKENS, MOE_MAX_SEQUENCES = 1 << 20, 65535
SCORES = {"sigmoid": MOE_SCORE_SIGMOID, "softmax": MOE_SCORE_SOFTMAX}


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: status {status} ({status_string(status)})")
        self.status = status


class moe_bank(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("base", ctypes.c_void_p), ("expert_stride", ctypes.c_int64),
                ("offset", ctypes.c_int64 * MOE_NUM_TENSORS)]


class moe_latent_layer(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("w_router", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("norm_gamma", ctypes.c_void_p),
                ("norm_eps", ctypes.c_float), ("w_up", ctypes.c_void_p),
                ("routed", moe_bank), ("shared", moe_bank)]


class moe_quant_matrix(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("group", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32), ("codes", ctypes.c_void_p),
                ("code_pitch", ctypes.c_int64), ("scales", ctypes.c_void_p),
                ("scale_pitch", ctypes.c_int64), ("zeros", ctypes.c_void_p),
                ("zero_pitch", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run __graft_entry__.build() "
                               "(or routed_expert_fp4_amd.build.build_library()) first")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        f32 = ctypes.c_float
        sig = {
            "moe_version": ([], i32),
            "moe_status_string": ([i32], ctypes.c_char_p),
            "moe_bank_layout": ([i32, i32, i32, P, P], i32),
            "moe_workspace_size": ([i32, i32, i32, i32, i32], sz),
            "moe_workspace_init": ([P, sz, P], i32),
            "moe_route": ([P, P, P, i32, i32, i32, i32, P, P, P, sz, P], i32),
            "moe_expert_fwd": ([P, P, i32, i32, P, P, P, P, sz, P], i32),
            "moe_layer_fwd": ([P, P, P, i32, i32, P, P, P, P, sz, P], i32),
            "moe_dequant": ([P, i32, i32, P, P], i32),
            "moe_latent_workspace_size": ([P, i32, i32], sz),
            "moe_latent_layer_fwd": ([P, P, i32, i32, P, P, P, P, sz, P], i32),
            "moe_mx_mma_workspace_size": ([P, i32, i32, i32], sz),
            "moe_expert_fwd_mx_mma": ([P, P, i32, i32, P, P, P, i32, P, sz, P], i32),
            "moe_layer_fwd_noalloc": ([P, P, P, i32, i32, P, P, P, P, P], i32),
            "moe_quant_workspace_size": ([P, i32, i32], sz),
            "moe_quant_linear": ([P, i32, P, i64, i32, P, i64, i32, P, sz, P], i32),
            "moe_expert_counts": ([P, i32, i32, i32, P, i32, P, P, P, i32, P], i32),
            "moe_balance_workspace_size": ([i32, i32, i32], sz),
            "moe_balance_fwd": ([P, P, i32, i32, i32, P, i32, P, i32, f32, P, P, P, P, P, sz, P], i32),
            "moe_balance_bwd": ([P, P, P, i32, i32, i32, P, i32, P, i32, f32, P, P, i32, P], i32),
            "moe_route_bwd": ([P, P, P, i32, i32, i32, P, P, i32, P], i32),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def _check(fn: str, status: int) -> None:
    if status != MOE_OK:
        raise MoeError(fn, status)


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t, dtype=None, shape=None, name="tensor"):
    """Device pointer of a contiguous CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return ctypes.c_void_p(t.data_ptr())


# ---------------------------------------------------------------------------
# Bank layout and workspace
# ---------------------------------------------------------------------------
def moe_version() -> int:
    return lib().moe_version()


def moe_bank_layout(fmt: int, hidden: int, inter: int):
    """(offsets[7], expert_stride) of the library's preferred record layout."""
    off = (ctypes.c_int64 * MOE_NUM_TENSORS)()
    stride = ctypes.c_int64()
    _check("moe_bank_layout", lib().moe_bank_layout(fmt, hidden, inter, off, ctypes.byref(stride)))
    return list(off), stride.value


def moe_workspace_size(num_experts: int, hidden: int, inter: int, top_k: int, C: int) -> int:
    n = lib().moe_workspace_size(num_experts, hidden, inter, top_k, C)
    if n == 0:
        raise MoeError("moe_workspace_size", MOE_ERR_UNSUPPORTED)
    return n


def moe_workspace_init(ws, stream=None) -> None:
    _check("moe_workspace_init", lib().moe_workspace_init(_ptr(ws, name="ws"), ws.numel() * ws.element_size(), _stream(stream)))


class Bank:
    """An expert bank held in one device allocation, with its moe_bank struct."""

    def __init__(self, fmt: int, num_experts: int, hidden: int, inter: int, device="cuda",
                 storage=None):
        import torch
        self.fmt, self.E, self.H, self.I = fmt, num_experts, hidden, inter
        self.offsets, self.stride = moe_bank_layout(fmt, hidden, inter)
        nbytes = self.stride * num_experts
        self.storage = (torch.empty(nbytes, dtype=torch.uint8, device=device)
                        if storage is None else storage)
        if self.storage.numel() < nbytes:
            raise ValueError("bank storage too small")
        self.struct = moe_bank(fmt, num_experts, hidden, inter, self.storage.data_ptr(),
                               self.stride, (ctypes.c_int64 * MOE_NUM_TENSORS)(*self.offsets))

    def tensor_view(self, expert: int, tensor: int, nbytes: int):
        base = expert * self.stride + self.offsets[tensor]
        return self.storage[base: base + nbytes]


def _bank(b):
    return ctypes.byref(b.struct if isinstance(b, Bank) else b)


class Workspace:
    """A zero-initialised device workspace sized for (E, H, I, k, C)."""

    def __init__(self, num_experts, hidden, inter, top_k, C, device="cuda", stream=None):
        import torch
        n = moe_workspace_size(num_experts, hidden, inter, top_k, C)
        self.tensor = torch.empty((n + 255) // 256 * 256 // 4, dtype=torch.int32, device=device)
        moe_workspace_init(self.tensor, stream)

    @property
    def ptr(self):
        return ctypes.c_void_p(self.tensor.data_ptr())

    @property
    def nbytes(self):
        return self.tensor.numel() * 4


# ---------------------------------------------------------------------------
# The path
# ---------------------------------------------------------------------------
def moe_route(x, w_router, logits, C, H, E, k, topk_idx, topk_w, ws: Workspace, stream=None):
    """Router + top-k.  x None -> logits-in mode (logits is read)."""
    import torch
    _check("moe_route", lib().moe_route(
        _ptr(x, torch.float32, (C, H), "x"), _ptr(w_router, torch.float32, (E, H), "w_router"),
        _ptr(logits, torch.float32, (C, E), "logits"), C, H, E, k,
        _ptr(topk_idx, torch.int32, (C, k), "topk_idx"), _ptr(topk_w, torch.float32, (C, k), "topk_w"),
        ws.ptr, ws.nbytes, _stream(stream)))


def moe_expert_fwd(bank: Bank, x, C, k, topk_idx, topk_w, out, ws: Workspace, stream=None):
    import torch
    H = bank.H
    _check("moe_expert_fwd", lib().moe_expert_fwd(
        _bank(bank), _ptr(x, torch.float32, (C, H), "x"), C, k,
        _ptr(topk_idx, torch.int32, (C, k), "topk_idx"), _ptr(topk_w, torch.float32, (C, k), "topk_w"),
        _ptr(out, torch.float32, (C, H), "out"), ws.ptr, ws.nbytes, _stream(stream)))


def moe_layer_fwd(bank: Bank, w_router, x, C, k, out, topk_idx_out=None, topk_w_out=None,
                  ws: Workspace = None, stream=None):
    import torch
    H, E = bank.H, bank.E
    _check("moe_layer_fwd", lib().moe_layer_fwd(
        _bank(bank), _ptr(w_router, torch.float32, (E, H), "w_router"),
        _ptr(x, torch.float32, (C, H), "x"), C, k, _ptr(out, torch.float32, (C, H), "out"),
        _ptr(topk_idx_out, torch.int32, (C, k), "topk_idx_out"),
        _ptr(topk_w_out, torch.float32, (C, k), "topk_w_out"), ws.ptr, ws.nbytes, _stream(stream)))


def moe_layer_fwd_noalloc(bank: Bank, w_router, x, C, k, out, topk_idx_out=None,
                          topk_w_out=None, error_out=None, stream=None):
    """moe_layer_fwd on the library's own device array instead of a workspace."""
    import torch
    H, E = bank.H, bank.E
    _check("moe_layer_fwd_noalloc", lib().moe_layer_fwd_noalloc(
        _bank(bank), _ptr(w_router, torch.float32, (E, H), "w_router"),
        _ptr(x, torch.float32, (C, H), "x"), C, k, _ptr(out, torch.float32, (C, H), "out"),
        _ptr(topk_idx_out, torch.int32, (C, k), "topk_idx_out"),
        _ptr(topk_w_out, torch.float32, (C, k), "topk_w_out"),
        _ptr(error_out, torch.int32, (1,), "error_out"), _stream(stream)))


def moe_dequant(bank: Bank, expert: int, matrix: int, out, stream=None):
    import torch
    N, K = (bank.H, bank.I) if matrix == 2 else (bank.I, bank.H)
    _check("moe_dequant", lib().moe_dequant(_bank(bank), expert, matrix,
                                            _ptr(out, torch.float32, (N, K), "out"), _stream(stream)))


# ---------------------------------------------------------------------------
# Latent MoE layer (routed_down, routed experts, routed_norm, routed_up, shared)
# ---------------------------------------------------------------------------
class LatentLayer:
    """The device tensors of one latent MoE layer and its moe_latent_layer struct.
    w_router [E][H] fp32, w_down [L][H] and w_up [H][L] as int16/uint16 bf16
    bits, gamma [L] fp32; routed (hidden L) and shared (hidden H) are Banks."""

    def __init__(self, w_router, w_down, gamma, eps: float, w_up, routed: Bank, shared: Bank):
        import torch
        H, L = shared.H, routed.H
        _ptr(w_router, torch.float32, (routed.E, H), "w_router")
        if w_down.dtype not in (torch.int16, torch.uint16) or tuple(w_down.shape) != (L, H):
            raise ValueError(f"w_down must be bf16 bits of shape {(L, H)}")
        if w_up.dtype not in (torch.int16, torch.uint16) or tuple(w_up.shape) != (H, L):
            raise ValueError(f"w_up must be bf16 bits of shape {(H, L)}")
        _ptr(gamma, torch.float32, (L,), "gamma")
        self.keep = (w_router, w_down, gamma, w_up, routed, shared)
        self.H, self.L, self.E = H, L, routed.E
        self.struct = moe_latent_layer(H, w_router.data_ptr(), _ptr(w_down, name="w_down").value,
                                       gamma.data_ptr(), eps, _ptr(w_up, name="w_up").value,
                                       routed.struct, shared.struct)


class LatentWorkspace:
    def __init__(self, layer: LatentLayer, top_k: int, C: int, device="cuda", stream=None):
        import torch
        n = lib().moe_latent_workspace_size(ctypes.byref(layer.struct), top_k, C)
        if n == 0:
            raise MoeError("moe_latent_workspace_size", MOE_ERR_UNSUPPORTED)
        self.tensor = torch.empty((n + 255) // 256 * 256 // 4, dtype=torch.int32, device=device)
        moe_workspace_init(self.tensor, stream)

    @property
    def ptr(self):
        return ctypes.c_void_p(self.tensor.data_ptr())

    @property
    def nbytes(self):
        return self.tensor.numel() * 4


def moe_latent_layer_fwd(layer: LatentLayer, x, C, k, out, topk_idx_out=None, topk_w_out=None,
                         ws: LatentWorkspace = None, stream=None):
    import torch
    H = layer.H
    _check("moe_latent_layer_fwd", lib().moe_latent_layer_fwd(
        ctypes.byref(layer.struct), _ptr(x, torch.float32, (C, H), "x"), C, k,
        _ptr(out, torch.float32, (C, H), "out"),
        _ptr(topk_idx_out, torch.int32, (C, k), "topk_idx_out"),
        _ptr(topk_w_out, torch.float32, (C, k), "topk_w_out"), ws.ptr, ws.nbytes, _stream(stream)))


# ---------------------------------------------------------------------------
# MXFP4 experts on the block-scaled FP4 matrix cores
# ---------------------------------------------------------------------------
class MxMmaWorkspace:
    def __init__(self, bank: Bank, top_k: int, C: int, terms: int, device="cuda"):
        import torch
        n = lib().moe_mx_mma_workspace_size(_bank(bank), top_k, C, terms)
        if n == 0:
            raise MoeError("moe_mx_mma_workspace_size", MOE_ERR_UNSUPPORTED)
        self.tensor = torch.empty((n + 255) // 256 * 256 // 4, dtype=torch.int32, device=device)

    @property
    def ptr(self):
        return ctypes.c_void_p(self.tensor.data_ptr())

    @property
    def nbytes(self):
        return self.tensor.numel() * 4


def moe_expert_fwd_mx_mma(bank: Bank, x, C, k, topk_idx, topk_w, out, terms: int,
                          ws: MxMmaWorkspace, stream=None):
    import torch
    H = bank.H
    _check("moe_expert_fwd_mx_mma", lib().moe_expert_fwd_mx_mma(
        _bank(bank), _ptr(x, torch.float32, (C, H), "x"), C, k,
        _ptr(topk_idx, torch.int32, (C, k), "topk_idx"), _ptr(topk_w, torch.float32, (C, k), "topk_w"),
        _ptr(out, torch.float32, (C, H), "out"), terms, ws.ptr, ws.nbytes, _stream(stream)))


# ---------------------------------------------------------------------------
# Dense matrices in 4-bit codes with group scales
# ---------------------------------------------------------------------------
class _Scratch:
    """A zero-initialised device workspace of `nbytes`."""

    def __init__(self, fn: str, nbytes: int, device, stream=None):
        import torch
        if nbytes == 0:
            raise MoeError(fn, MOE_ERR_UNSUPPORTED)
        self.tensor = torch.empty((nbytes + 255) // 256 * 64, dtype=torch.int32, device=device)
        self.nbytes, self.device = self.tensor.numel() * 4, self.tensor.get_device()
        with torch.cuda.device(self.tensor.device):
            moe_workspace_init(self.tensor, stream)


def _scratch(ws, kind, dev):
    """Pointer and bytes of a workspace of this kind on GPU `dev`: each keeps its
    own state between calls."""
    if not isinstance(ws, kind):
        raise ValueError(f"ws must be a {kind.__name__}, got {type(ws).__name__}")
    if ws.device != dev:
        raise ValueError(f"workspace must be on cuda:{dev}, got {ws.tensor.device}")
    return ws.tensor.data_ptr(), ws.nbytes


def _bad(t, dev, dtype, shape, name):
    """The first thing wrong with a tensor argument."""
    if not t.is_cuda:
        return ValueError(f"{name} must be a device tensor")
    if t.get_device() != dev:
        return ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if t.dtype != dtype:
        return ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        return ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return ValueError(f"{name} must have dense rows, got strides {t.stride()}")


def _dense(t, dev, dtype, shape, name):
    """Device pointer of a contiguous tensor of this type and shape on GPU `dev`."""
    if t.get_device() != dev or t.dtype != dtype or t.shape != shape or not t.is_contiguous() or dev < 0:
        raise _bad(t, dev, dtype, shape, name)
    return t.data_ptr()


def _maybe(t, dev, dtype, shape, name):
    """The same, or NULL for None."""
    return None if t is None else _dense(t, dev, dtype, shape, name)


def _rows(t, dev, dtype, shape, name):
    """(pointer, pitch in elements) of a matrix whose rows are dense."""
    if t.get_device() != dev or t.dtype != dtype or t.shape != shape or dev < 0:
        raise _bad(t, dev, dtype, shape, name)
    pitch, step = t.stride()
    if (step != 1 and shape[1] > 1) or (pitch < shape[1] and shape[0] > 1):
        raise _bad(t, dev, dtype, shape, name)
    return t.data_ptr(), pitch if shape[0] > 1 else shape[1]


_cuda = None      # torch's raw current stream of a GPU, and its current GPU


def _bind_cuda():
    """The two queries without the Python around them: a quarter of a
    microsecond less per call."""
    global _cuda
    import torch
    _cuda = (getattr(torch._C, "_cuda_getCurrentRawStream", None) or
             (lambda dev: torch.cuda.current_stream(dev).cuda_stream),
             getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device)
    return _cuda


def _launch(fn, dev, stream, *args):
    """Calls an entry point on GPU `dev` and its stream (None: the current
    one), whichever GPU is current."""
    raw_stream, current = _cuda or _bind_cuda()
    if stream is None:
        handle = raw_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"the stream must be of cuda:{dev}, got {stream.device}")
    else:
        handle = stream.cuda_stream
    f = getattr(_lib or lib(), fn)
    if current() == dev:
        status = f(*args, handle)
    else:
        import torch
        with torch.cuda.device(dev):
            status = f(*args, handle)
    if status != MOE_OK:
        raise MoeError(fn, status)


def _moe_dtype(dtype):
    import torch
    d = {torch.float32: MOE_DT_F32, torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16}.get(dtype)
    if d is None:
        raise ValueError(f"type must be float32, bfloat16 or float16, got {dtype}")
    return d


class QuantMatrix:
    """The device tensors of one dense 4-bit matrix [N][K] and its
    moe_quant_matrix struct: W[n][k] = scales[n][k // group] *
    (code[n][k] - zeros[n][k // group]), zeros 8 where none are given.
    codes [N][>= K / 2] uint8 (element 2j in the low half of byte j), rows
    16-byte aligned; scales [N][>= K / group] fp32, bf16 or fp16; zeros uint8."""

    def __init__(self, codes, scales, K: int, group: int, zeros=None):
        import torch
        if codes.dim() != 2 or K < 1 or group < 1:
            raise ValueError(f"codes must be a matrix and K, group >= 1, got {tuple(codes.shape)}, {K}, {group}")
        dev = codes.get_device()
        N, ng = codes.shape[0], -(-K // group)
        units = -(-K // 32)
        _, pitch = _rows(codes, dev, torch.uint8, codes.shape, "codes")
        if N == 1:
            pitch = 16 * units                       # no second row to be a pitch away
        if codes.shape[1] < -(-K // 2):
            raise ValueError(f"codes must have {-(-K // 2)} bytes a row, got {codes.shape[1]}")
        # the last row's last 16-byte unit is read whole
        have = codes.untyped_storage().nbytes() - codes.storage_offset()
        if have < (N - 1) * pitch + 16 * units:
            raise ValueError("codes: the last row must be readable up to a multiple of 16 bytes")
        self.tables = []
        for t, name, dtype in ((scales, "scales", scales.dtype), (zeros, "zeros", torch.uint8)):
            if t is None:
                self.tables += [None, 0]
                continue
            if t.dim() != 2 or t.shape[0] != N or t.shape[1] < ng:
                raise ValueError(f"{name} must have shape {(N, ng)}, got {tuple(t.shape)}")
            self.tables += _rows(t, dev, dtype, t.shape, name)
        self.N, self.K, self.group, self.device = N, K, group, dev
        self.keep = (codes, scales, zeros)
        self.struct = moe_quant_matrix(N, K, group, _moe_dtype(scales.dtype), codes.data_ptr(), pitch,
                                       *self.tables)
        self.ref = ctypes.byref(self.struct)


class QuantWorkspace(_Scratch):
    def __init__(self, matrix: QuantMatrix, C: int, dtype, stream=None):
        n = lib().moe_quant_workspace_size(matrix.ref, _moe_dtype(dtype), C)
        super().__init__("moe_quant_workspace_size", n, f"cuda:{matrix.device}", stream)


def moe_quant_linear(matrix: QuantMatrix, x, C, y, ws: QuantWorkspace, accumulate=False, stream=None):
    """y [C][N] = x [C][K] W^T (or y += with accumulate); x and y of one type,
    rows dense, any pitch."""
    dev, dtype = matrix.device, x.dtype
    xp, xs = _rows(x, dev, dtype, (C, matrix.K), "x")
    yp, ys = _rows(y, dev, dtype, (C, matrix.N), "y")
    _launch("moe_quant_linear", dev, stream, matrix.ref, _moe_dtype(dtype), xp, xs, C, yp, ys, accumulate,
            *_scratch(ws, QuantWorkspace, dev))


# ---------------------------------------------------------------------------
# Router load: counts, the balance loss, and the gradients of a router
# ---------------------------------------------------------------------------
def _score(score):
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    return SCORES[score]


def moe_expert_counts(topk_idx, C, E, k, counts, tokens=None, seq_offsets=None, S=1, token_mask=None,
                      accumulate=False, stream=None):
    """counts [S][E] (and tokens [S]) int32 of a selection topk_idx [C][k]."""
    import torch
    dev, i32 = topk_idx.get_device(), torch.int32
    _launch("moe_expert_counts", dev, stream, _dense(topk_idx, dev, i32, (C, k), "topk_idx"), C, k, E,
            _maybe(seq_offsets, dev, i32, (S + 1,), "seq_offsets"), S,
            _maybe(token_mask, dev, torch.uint8, (C,), "token_mask"),
            _dense(counts, dev, i32, (S, E), "counts"), _maybe(tokens, dev, i32, (S,), "tokens"),
            accumulate)


class BalanceWorkspace(_Scratch):
    def __init__(self, C: int, E: int, S: int = 1, device="cuda", stream=None):
        super().__init__("moe_balance_workspace_size", lib().moe_balance_workspace_size(C, E, S),
                         device, stream)


def moe_balance_fwd(logits, topk_idx, C, E, k, alpha, counts, tokens, probs, loss,
                    ws: BalanceWorkspace, score="sigmoid", seq_offsets=None, S=1, token_mask=None,
                    stream=None):
    """The balance loss of a selection, with its counts [S][E], tokens [S] and
    mean shares probs [S][E]."""
    import torch
    dev, i32, f32 = logits.get_device(), torch.int32, torch.float32
    _launch("moe_balance_fwd", dev, stream, _dense(logits, dev, f32, (C, E), "logits"),
            _dense(topk_idx, dev, i32, (C, k), "topk_idx"), C, k, E,
            _maybe(seq_offsets, dev, i32, (S + 1,), "seq_offsets"), S,
            _maybe(token_mask, dev, torch.uint8, (C,), "token_mask"), _score(score), alpha,
            _dense(counts, dev, i32, (S, E), "counts"), _dense(tokens, dev, i32, (S,), "tokens"),
            _dense(probs, dev, f32, (S, E), "probs"), _dense(loss, dev, f32, (1,), "loss"),
            *_scratch(ws, BalanceWorkspace, dev))


def moe_balance_bwd(logits, counts, tokens, C, E, k, alpha, grad_loss, dlogits, score="sigmoid",
                    seq_offsets=None, S=1, token_mask=None, accumulate=False, stream=None):
    """dlogits [C][E] of the balance loss, from what moe_balance_fwd wrote and
    grad_loss [1]."""
    import torch
    dev, i32, f32 = logits.get_device(), torch.int32, torch.float32
    _launch("moe_balance_bwd", dev, stream, _dense(logits, dev, f32, (C, E), "logits"),
            _dense(counts, dev, i32, (S, E), "counts"), _dense(tokens, dev, i32, (S,), "tokens"), C, k, E,
            _maybe(seq_offsets, dev, i32, (S + 1,), "seq_offsets"), S,
            _maybe(token_mask, dev, torch.uint8, (C,), "token_mask"), _score(score), alpha,
            _dense(grad_loss, dev, f32, (1,), "grad_loss"), _dense(dlogits, dev, f32, (C, E), "dlogits"),
            accumulate)


def moe_route_bwd(logits, topk_idx, topk_dw, C, E, k, dlogits, token_mask=None, accumulate=False,
                  stream=None):
    """dlogits [C][E] from topk_dw [C][k], the gradient of moe_route's weights."""
    import torch
    dev, f32 = logits.get_device(), torch.float32
    _launch("moe_route_bwd", dev, stream, _dense(logits, dev, f32, (C, E), "logits"),
            _dense(topk_idx, dev, torch.int32, (C, k), "topk_idx"),
            _dense(topk_dw, dev, f32, (C, k), "topk_dw"), C, k, E,
            _maybe(token_mask, dev, torch.uint8, (C,), "token_mask"),
            _dense(dlogits, dev, f32, (C, E), "dlogits"), accumulate)
