"""Python binding of the block-quantized MoE gather-qmm library (``libbq.so``).

Argument marshalling only: every function forwards device pointers of
PyTorch tensors and the current CUDA stream to the C ABI declared in
``include/bq.h``.  All arithmetic runs in the library's CUDA kernels; there
is no CPU fallback.  Importing this package fails when the library has not
been built (``python block_quantized_moe_gather_gb300/build.py``).
"""
from __future__ import annotations

import ctypes
import os
import struct
from ctypes import POINTER, c_char_p, c_float, c_int32, c_int64, c_size_t, c_uint64, c_void_p

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python block_quantized_moe_gather_gb300/build.py`")
_lib = ctypes.CDLL(LIB_PATH)

# ---------------------------------------------------------------- constants
OK = 0
FMT_Q8_0, FMT_Q2_K, FMT_INT4_G64, FMT_MXFP4, FMT_FP8_B128 = 1, 2, 3, 4, 5
FMT_BY_NAME = {"q8_0": FMT_Q8_0, "q2_k": FMT_Q2_K, "int4": FMT_INT4_G64, "mxfp4": FMT_MXFP4,
               "fp8_b128": FMT_FP8_B128}
DEV_OK, DEV_BAD_EXPERT_ID, DEV_WAIT_TIMEOUT, DEV_SCALE_RANGE, DEV_BAD_ROW = 0, 1, 2, 3, 4
DT_F32, DT_F16, DT_BF16 = 0, 1, 2
STATUS_NAMES = {0: "BQ_OK", 1: "BQ_ERR_NULL", 2: "BQ_ERR_SHAPE", 3: "BQ_ERR_ALIGN", 4: "BQ_ERR_FORMAT",
                5: "BQ_ERR_WORKSPACE", 6: "BQ_ERR_CUDA", 7: "BQ_ERR_DEVICE", 8: "BQ_ERR_ARCH"}


class QWeightC(ctypes.Structure):
    _fields_ = [("fmt", c_int32), ("n_mats", c_int32), ("n", c_int32), ("k", c_int32),
                ("swiglu", c_int32), ("reserved", c_int32), ("data", c_void_p)]


class MoEDescC(ctypes.Structure):
    _fields_ = [("T", c_int32), ("hidden", c_int32), ("inter", c_int32), ("n_experts", c_int32),
                ("topk", c_int32), ("scoring", c_int32), ("w_gate_up", QWeightC), ("w_down", QWeightC),
                ("shared_gate_up", POINTER(QWeightC)), ("shared_down", POINTER(QWeightC)),
                ("route_scale", c_float), ("reserved", c_int32)]


# Host structs that are made anew for every call, as bytes in the layout of bq.h (a ctypes.Structure of that many fields
# takes 1 us to make, a tenth of a small call; the bytes of an object lie on 16-byte boundaries).
_EPILOGUE = struct.Struct("if2Pq")                  # bq_epilogue: act, scale, bias, residual, ldr
_RESIDUAL_NORM_DESC = struct.Struct("9i3f3Pq")      # bq_residual_norm_desc, in its order


_SIGS = {
    "bq_status_string": (c_char_p, [c_int32]),
    "bq_last_error": (c_char_p, []),
    "bq_device_status": (c_int32, [c_void_p, POINTER(c_int32)]),
    "bq_gguf_dequant_q8_0": (c_int32, [c_void_p, c_int64, c_void_p, c_void_p]),
    "bq_gguf_dequant_q2_k": (c_int32, [c_void_p, c_int64, c_void_p, c_void_p]),
    "bq_dequant_mxfp4": (c_int32, [c_void_p, c_int64, c_void_p, c_void_p]),
    "bq_dequant_fp8_b128": (c_int32, [c_void_p, c_void_p, c_int64, c_int64, c_void_p, c_void_p]),
    "bq_qweight_bytes": (c_size_t, [c_int32, c_int32, c_int32, c_int32]),
    "bq_repack_q8_0": (c_int32, [c_void_p, POINTER(QWeightC), c_void_p]),
    "bq_repack_q2_k": (c_int32, [c_void_p, POINTER(QWeightC), c_void_p]),
    "bq_repack_int4": (c_int32, [c_void_p, c_void_p, c_void_p, POINTER(QWeightC), c_void_p]),
    "bq_repack_mxfp4": (c_int32, [c_void_p, POINTER(QWeightC), c_void_p]),
    "bq_repack_fp8_b128": (c_int32, [c_void_p, c_void_p, POINTER(QWeightC), c_void_p]),
    "bq_qmm": (c_int32, [c_void_p, c_int32, POINTER(QWeightC), c_void_p, c_void_p]),
    "bq_moe_route": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p, c_void_p]),
    "bq_moe_route_scored": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int32, c_float, c_void_p,
                                      c_void_p, c_void_p]),
    "bq_moe_permute_workspace_bytes": (c_size_t, [c_int32, c_int32, c_int32]),
    "bq_moe_permute": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_size_t, c_void_p]),
    "bq_moe_workspace_bytes": (c_size_t, [POINTER(MoEDescC)]),
    "bq_moe_permute_noalloc": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p, c_void_p,
                                         c_void_p, c_void_p, c_void_p]),
    "bq_set_stage_events": (c_int32, [c_int32, c_void_p, c_void_p]),
    "bq_rmsnorm": (c_int32, [c_void_p, c_int32, c_int32, c_void_p, c_float, c_void_p, c_void_p]),
    "bq_rmsnorm_qmm": (c_int32, [c_void_p, c_int32, c_void_p, c_float, POINTER(QWeightC), c_void_p, c_void_p,
                                 c_void_p]),
    "bq_moe_hidden_workspace_bytes": (c_size_t, [POINTER(MoEDescC)]),
    "bq_moe_gather_qmm_hidden": (c_int32, [POINTER(MoEDescC), POINTER(QWeightC), c_void_p, c_void_p, c_float,
                                           c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "bq_launch_count": (c_uint64, []),
    "bq_test_set_wait_probe": (c_int32, [c_int32, c_uint64]),
    "bq_moe_gather_qmm": (c_int32, [POINTER(MoEDescC), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                    c_size_t, c_void_p]),
    "bq_moe_dispatch": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_int64, c_void_p, c_int32, c_void_p, c_int64,
                                  c_void_p]),
    "bq_moe_dispatch_backward": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_int64, c_void_p, c_int32, c_void_p,
                                           c_int64, c_void_p]),
    "bq_moe_combine": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_int64, c_void_p, c_void_p, c_int32, c_int32,
                                 c_void_p, c_int64, c_void_p]),
    "bq_moe_combine_backward": (c_int32, [c_void_p, c_int64, c_void_p, c_int64, c_int32, c_int32, c_int32, c_void_p,
                                          c_void_p, c_int32, c_void_p, c_int64, c_void_p, c_void_p]),
    "bq_quant_fp8_b128": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_int64, c_void_p, c_void_p, c_void_p,
                                    c_void_p]),
    "bq_moe_dispatch_fp8_b128": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_int64, c_void_p, c_int32, c_void_p,
                                           c_void_p, c_void_p]),
    "bq_mm_fp8_b128": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_int32, c_int32, c_void_p,
                                 c_int32, c_int64, c_void_p]),
    "bq_moe_mm_fp8_b128": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_int32,
                                     c_int32, c_int32, c_void_p, c_int32, c_int64, c_void_p]),
    "bq_mm_fp8_b128_epilogue": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_int32,
                                          c_char_p, c_void_p, c_int32, c_int64, c_void_p]),
    "bq_moe_mm_fp8_b128_epilogue": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_void_p,
                                              c_int32, c_int32, c_char_p, c_void_p, c_int32, c_int64,
                                              c_void_p]),
    "bq_residual_norm": (c_int32, [c_char_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64,
                                   c_void_p, c_int64, c_void_p]),
    "bq_residual_norm_backward_workspace_bytes": (c_size_t, [c_int32, c_int32]),
    "bq_residual_norm_backward": (c_int32, [c_char_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p,
                                            c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p,
                                            c_void_p, c_void_p, c_int64, c_void_p, c_size_t, c_void_p]),
    "bq_moe_balance_workspace_bytes": (c_size_t, [c_int32, c_int32, c_int32]),
    "bq_moe_balance_loss": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_int32, c_int32, c_void_p,
                                      c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "bq_moe_route_backward_workspace_bytes": (c_size_t, [c_int32, c_int32]),
    "bq_moe_route_backward": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_int32, c_int32, c_float,
                                        c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_int32, c_void_p,
                                        c_void_p, c_size_t, c_void_p]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class BQError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str | None = None):
        self.status = status
        if msg is None:
            msg = _lib.bq_last_error().decode(errors="replace")
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {msg}")


def _check(status: int, where: str):
    if status != OK:
        raise BQError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        if _DT is None:
            _load_torch()
        return _get_stream(_get_device())
    return stream.cuda_stream


def status_string(s: int) -> str:
    return _lib.bq_status_string(s).decode()


def last_error() -> str:
    return _lib.bq_last_error().decode()


def device_status(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status code."""
    code = c_int32(0)
    st = _lib.bq_device_status(_stream(stream), ctypes.byref(code))
    if st not in (OK, 7):
        raise BQError(st, "bq_device_status")
    return code.value


# ---------------------------------------------------------------- dequant
def gguf_dequant_q8_0(blocks, out, stream=None):
    """blocks: uint8 device tensor of n*34 bytes; out: fp32 device tensor of n*32."""
    n = blocks.numel() // 34
    _check(_lib.bq_gguf_dequant_q8_0(_ptr(blocks), n, _ptr(out), _stream(stream)), "bq_gguf_dequant_q8_0")
    return out


def gguf_dequant_q2_k(blocks, out, stream=None):
    n = blocks.numel() // 84
    _check(_lib.bq_gguf_dequant_q2_k(_ptr(blocks), n, _ptr(out), _stream(stream)), "bq_gguf_dequant_q2_k")
    return out


def dequant_mxfp4(blocks, out, stream=None):
    """blocks: uint8 device tensor of n*17 bytes; out: fp32 device tensor of n*32."""
    n = blocks.numel() // 17
    _check(_lib.bq_dequant_mxfp4(_ptr(blocks), n, _ptr(out), _stream(stream)), "bq_dequant_mxfp4")
    return out


def dequant_fp8_b128(weight, scales, out, stream=None):
    """weight: uint8 device tensor [n, k] (e4m3 bytes); scales: fp32 [ceil(n/128), ceil(k/128)];
    out: fp32 [n, k]."""
    n, k = weight.shape
    _check(_lib.bq_dequant_fp8_b128(_ptr(weight), _ptr(scales), n, k, _ptr(out), _stream(stream)),
           "bq_dequant_fp8_b128")
    return out


# ---------------------------------------------------------------- weights
def qweight_bytes(fmt: int, n_mats: int, n: int, k: int) -> int:
    return int(_lib.bq_qweight_bytes(fmt, n_mats, n, k))


class QWeight:
    """A repacked quantised weight stack [n_mats][n][k] held in a device
    uint8 tensor (``buf``), plus the C descriptor pointing at it."""

    def __init__(self, fmt: int, n_mats: int, n: int, k: int, swiglu: bool = False, device="cuda"):
        import torch
        nbytes = qweight_bytes(fmt, n_mats, n, k)
        if nbytes == 0:
            raise BQError(2, f"QWeight(fmt={fmt}, {n_mats}x{n}x{k})")
        # 256-byte alignment: the caching allocator returns 512-byte aligned blocks
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.fmt, self.n_mats, self.n, self.k, self.swiglu = fmt, n_mats, n, k, int(swiglu)
        self.c = QWeightC(fmt, n_mats, n, k, int(swiglu), 0, self.buf.data_ptr())

    @property
    def nbytes(self) -> int:
        return self.buf.numel()


def repack_q8_0(blocks, w: QWeight, stream=None) -> QWeight:
    _check(_lib.bq_repack_q8_0(_ptr(blocks), ctypes.byref(w.c), _stream(stream)), "bq_repack_q8_0")
    return w


def repack_q2_k(blocks, w: QWeight, stream=None) -> QWeight:
    _check(_lib.bq_repack_q2_k(_ptr(blocks), ctypes.byref(w.c), _stream(stream)), "bq_repack_q2_k")
    return w


def repack_int4(words, scales, biases, w: QWeight, stream=None) -> QWeight:
    _check(_lib.bq_repack_int4(_ptr(words), _ptr(scales), _ptr(biases), ctypes.byref(w.c), _stream(stream)),
           "bq_repack_int4")
    return w


def repack_mxfp4(blocks, w: QWeight, stream=None) -> QWeight:
    _check(_lib.bq_repack_mxfp4(_ptr(blocks), ctypes.byref(w.c), _stream(stream)), "bq_repack_mxfp4")
    return w


def repack_fp8_b128(weight, scales, w: QWeight, stream=None) -> QWeight:
    _check(_lib.bq_repack_fp8_b128(_ptr(weight), _ptr(scales), ctypes.byref(w.c), _stream(stream)),
           "bq_repack_fp8_b128")
    return w


# ---------------------------------------------------------------- compute
def qmm(x, w: QWeight, y, stream=None):
    """y[m][n] = x[m][k] W^T; x fp16 [m, k], y fp32 [m, n] (device)."""
    m = x.shape[0] if x.dim() == 2 else 1
    _check(_lib.bq_qmm(_ptr(x), m, ctypes.byref(w.c), _ptr(y), _stream(stream)), "bq_qmm")
    return y


def moe_route(logits, bias, k: int, ids, weights, stream=None):
    t, e = logits.shape
    _check(_lib.bq_moe_route(_ptr(logits), _ptr(bias), t, e, k, _ptr(ids), _ptr(weights), _stream(stream)),
           "bq_moe_route")


# bq_scoring
SCORE_SOFTMAX, SCORE_SOFTMAX_THEN_BIAS, SCORE_SQRTSOFTPLUS = 0, 1, 2
SCORING_BY_NAME = {"softmax": SCORE_SOFTMAX, "softmax_then_bias": SCORE_SOFTMAX_THEN_BIAS,
                   "sqrtsoftplus": SCORE_SQRTSOFTPLUS}


def moe_route_scored(logits, bias, k: int, scoring: int, scale: float, ids, weights, stream=None):
    t, e = logits.shape
    _check(_lib.bq_moe_route_scored(_ptr(logits), _ptr(bias), t, e, k, scoring, scale, _ptr(ids), _ptr(weights),
                                    _stream(stream)),
           "bq_moe_route_scored")


def moe_permute_workspace_bytes(t: int, k: int, e: int) -> int:
    return int(_lib.bq_moe_permute_workspace_bytes(t, k, e))


def moe_permute(ids, n_experts: int, counts, offsets, perm_token, perm_slot, inv, workspace, stream=None):
    t, k = ids.shape
    _check(_lib.bq_moe_permute(_ptr(ids), t, k, n_experts, _ptr(counts), _ptr(offsets), _ptr(perm_token),
                               _ptr(perm_slot), _ptr(inv), _ptr(workspace), workspace.numel(), _stream(stream)),
           "bq_moe_permute")


STAGE_ROUTE_PERMUTE, STAGE_GATE_UP, STAGE_DOWN, STAGE_SHARED, STAGE_COMBINE, STAGE_NORM_ROUTER = range(6)


def set_stage_events(stage: int, start=None, stop=None):
    """Have later layer calls record `start`/`stop` (torch.cuda.Event, already
    recorded once so that they exist) around one stage; None clears."""
    h = (lambda ev: None if ev is None else ctypes.c_void_p(ev.cuda_event))
    _check(_lib.bq_set_stage_events(stage, h(start), h(stop)), "bq_set_stage_events")


def launch_count() -> int:
    return int(_lib.bq_launch_count())


def test_set_wait_probe(skip_weight_copies: bool, wait_limit_ns: int = 0, odd_parts_only: bool = False):
    """Test hook: GEMM launches that follow take `wait_limit_ns` as the bound of
    their barrier waits and, with `skip_weight_copies`, issue no weight copies
    (so those waits run out), with `odd_parts_only` only in the odd parts of an
    FP8 product's K split; (False, 0) restores the defaults."""
    skip = int(bool(skip_weight_copies)) | (2 if odd_parts_only else 0)
    _check(_lib.bq_test_set_wait_probe(skip, int(wait_limit_ns)), "bq_test_set_wait_probe")


def moe_permute_noalloc(ids, n_experts: int, counts, offsets, perm_token, perm_slot, inv, stream=None):
    """bq_moe_permute without a workspace: for callers that cannot allocate
    device memory at call time.  Scratch is a fixed array built into the
    library (limit: ceil(T*k/256) * E <= 65536); calls that overlap on the
    GPU race on it."""
    t, k = ids.shape
    _check(_lib.bq_moe_permute_noalloc(_ptr(ids), t, k, n_experts, _ptr(counts), _ptr(offsets), _ptr(perm_token),
                                       _ptr(perm_slot), _ptr(inv), _stream(stream)),
           "bq_moe_permute_noalloc")


class MoELayer:
    """Descriptor of one MoE layer over repacked weights (host struct)."""

    def __init__(self, t: int, hidden: int, inter: int, n_experts: int, topk: int, w_gate_up: QWeight,
                 w_down: QWeight, shared_gate_up: QWeight | None = None, shared_down: QWeight | None = None,
                 scoring: int = 0, route_scale: float = 1.0):
        self.weights = (w_gate_up, w_down, shared_gate_up, shared_down)  # keep buffers alive
        self._s_gu = shared_gate_up.c if shared_gate_up else None
        self._s_d = shared_down.c if shared_down else None
        self.c = MoEDescC(t, hidden, inter, n_experts, topk, scoring, w_gate_up.c, w_down.c,
                          ctypes.pointer(self._s_gu) if self._s_gu else None,
                          ctypes.pointer(self._s_d) if self._s_d else None, route_scale, 0)

    def set_tokens(self, t: int):
        self.c.T = t

    def workspace_bytes(self) -> int:
        return int(_lib.bq_moe_workspace_bytes(ctypes.byref(self.c)))

    def hidden_workspace_bytes(self) -> int:
        """Workspace of moe_gather_qmm_hidden (layer + normalised x + logits)."""
        return int(_lib.bq_moe_hidden_workspace_bytes(ctypes.byref(self.c)))


def moe_workspace_bytes(layer: MoELayer) -> int:
    return layer.workspace_bytes()


def moe_gather_qmm(layer: MoELayer, x, router_logits, logit_bias, y, workspace, stream=None):
    _check(_lib.bq_moe_gather_qmm(ctypes.byref(layer.c), _ptr(x), _ptr(router_logits), _ptr(logit_bias),
                                  _ptr(y), _ptr(workspace), workspace.numel(), _stream(stream)),
           "bq_moe_gather_qmm")
    return y


# ---------------------------------------------------------------- RMSNorm, fused
def rmsnorm(h, gamma, eps: float, x, stream=None):
    """x = gamma * h / sqrt(mean(h^2) + eps) per row; h, x fp16 [T, H], gamma fp16 [H]."""
    t, hdim = h.shape
    _check(_lib.bq_rmsnorm(_ptr(h), t, hdim, _ptr(gamma), eps, _ptr(x), _stream(stream)), "bq_rmsnorm")
    return x


def rmsnorm_qmm(h, gamma, eps: float, w: QWeight, y, x_out=None, stream=None):
    """y = W rmsnorm(h) (fp32 [m, n]); x_out (fp16 [m, k]) receives the normalised
    rows (required for m > 8)."""
    m = h.shape[0]
    _check(_lib.bq_rmsnorm_qmm(_ptr(h), m, _ptr(gamma), eps, ctypes.byref(w.c), _ptr(x_out), _ptr(y),
                               _stream(stream)),
           "bq_rmsnorm_qmm")
    return y


def moe_gather_qmm_hidden(layer: MoELayer, router: QWeight, hidden, gamma, eps: float, logit_bias, y, workspace,
                          stream=None):
    """The MoE layer from hidden states: RMSNorm + router matmul, then moe_gather_qmm."""
    _check(_lib.bq_moe_gather_qmm_hidden(ctypes.byref(layer.c), ctypes.byref(router.c), _ptr(hidden), _ptr(gamma),
                                         eps, _ptr(logit_bias), _ptr(y), _ptr(workspace), workspace.numel(),
                                         _stream(stream)),
           "bq_moe_gather_qmm_hidden")
    return y


# ---------------------------------------------------------------- rows by expert, FP8 rows and products
# These calls read shapes, strides and types from their tensors, so the tensors
# are checked here: a call that does not fit raises BQError and launches nothing.
# A small call lasts a few microseconds on the GPU, so the checks read each
# attribute once, and torch (imported lazily by this package) is looked up once.
_DT = None          # torch dtype -> bq_dtype
_KINDS = None       # _dense's kinds -> the torch dtypes they take
_get_device = None  # ordinal of the current CUDA device
_get_stream = None  # handle of a device's current stream


def _load_torch():
    global _DT, _KINDS, _get_device, _get_stream
    import torch
    _DT = {torch.float32: DT_F32, torch.float16: DT_F16, torch.bfloat16: DT_BF16}
    _KINDS = {"f32": (torch.float32,), "i32": (torch.int32,), "fp8": (torch.float8_e4m3fn, torch.uint8)}
    # the private calls return plain numbers; a torch.cuda.Stream object alone costs 3 us to make
    _get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _get_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)


def _refuse(status: int, where: str, msg: str):
    raise BQError(status, where, msg)


def _on_stream(where: str, stream, first, *tensors):
    """Handle of `stream` (None: the current one), after checking that every tensor
    is on the current CUDA device, the one the stream belongs to."""
    if _DT is None:
        _load_torch()
    device = first.get_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            _refuse(2, where, f"tensors are on {first.device} and {t.device}")
    if device < 0:
        _refuse(2, where, f"a tensor is on {first.device}, not on a CUDA device")
    if device != _get_device():
        _refuse(2, where, f"the tensors are on cuda:{device}, the current device is cuda:{_get_device()}")
    return _get_stream(device) if stream is None else stream.cuda_stream


def _rows_of(where: str, what: str, t, rows=None, cols=None, dtype=None):
    """(pointer, bq_dtype, rows, cols, row stride) of a matrix whose rows are dense."""
    if _DT is None:
        _load_torch()
    shape = t.shape
    if rows is None:
        if len(shape) != 2:
            _refuse(2, where, f"{what} has shape {list(shape)}, expected [rows, columns]")
    elif shape != (rows, cols):
        _refuse(2, where, f"{what} has shape {list(shape)}, expected [{rows}, {cols}]")
    dt = _DT.get(t.dtype)
    if dt is None or (dtype is not None and dt != dtype):
        _refuse(4, where, f"{what} has type {t.dtype}")
    r, c = shape
    ld = c
    if not t.is_contiguous():
        ld, step = t.stride()
        if step != 1 and c > 1:
            _refuse(3, where, f"the rows of {what} are not contiguous (strides {(ld, step)})")
        if r <= 1:
            ld = c
    if r > 0x7fffffff or c > 0x7fffffff:
        _refuse(2, where, f"{what} has shape {list(shape)}")
    return t.data_ptr(), dt, r, c, ld


def _dense(where: str, what: str, t, shape, kind: str):
    """Pointer of a contiguous tensor of the given shape; kind: f32, i32 or fp8 (e4m3 bytes)."""
    if _DT is None:
        _load_torch()
    if t.dtype not in _KINDS[kind]:
        _refuse(4, where, f"{what} has type {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        _refuse(2, where, f"{what} has shape {list(t.shape)} and strides {tuple(t.stride())}, "
                          f"expected contiguous {list(shape)}")
    return t.data_ptr()


def _pairs(where: str, inv, t: int):
    """(pointer, k) of inv, int32 [T, k] or flat [T * k] as moe_permute writes it (T > 0)."""
    if _DT is None:
        _load_torch()
    if inv.dtype not in _KINDS["i32"]:
        _refuse(4, where, f"inv has type {inv.dtype}")
    shape = inv.shape
    if len(shape) == 2:
        k, rest = shape[1], shape[0] - t
    else:
        k, rest = divmod(shape[0], t) if len(shape) == 1 else (0, 1)
    if rest or not inv.is_contiguous():
        _refuse(2, where, f"inv has shape {list(shape)} and strides {tuple(inv.stride())} for {t} tokens")
    return inv.data_ptr(), k


def moe_dispatch(x, inv, xs, stream=None):
    """Rows into expert order: xs[inv[t][j]] = x[t].  x [T, H], xs [T*k, H] of one
    type (fp32, fp16, bf16), rows 16-byte aligned; inv int32 [T, k] or [T*k] from
    moe_permute (-1: a dropped pair)."""
    where = "bq_moe_dispatch"
    st = _on_stream(where, stream, x, inv, xs)
    px, dt, t, h, ldx = _rows_of(where, "x", x)
    if t == 0:
        return xs
    pi, k = _pairs(where, inv, t)
    po, _, _, _, ldo = _rows_of(where, "xs", xs, t * k, h, dt)
    _check(_lib.bq_moe_dispatch(px, dt, t, h, ldx, pi, k, po, ldo, st), where)
    return xs


def moe_dispatch_backward(dxs, inv, dx, stream=None):
    """Gradient of moe_dispatch: dx[t] = sum_j dxs[inv[t][j]] (fp32 sum, slot order)."""
    where = "bq_moe_dispatch_backward"
    st = _on_stream(where, stream, dxs, inv, dx)
    po, dt, t, h, ldo = _rows_of(where, "dx", dx)
    if t == 0:
        return dx
    pi, k = _pairs(where, inv, t)
    px, _, _, _, ldx = _rows_of(where, "dxs", dxs, t * k, h, dt)
    _check(_lib.bq_moe_dispatch_backward(px, dt, t, h, ldx, pi, k, po, ldo, st), where)
    return dx


def moe_combine(ys, inv, weights, y, accumulate: bool = False, stream=None):
    """Rows back in token order: y[t] = sum_j weights[t][j] * ys[inv[t][j]], with
    accumulate y[t] += that.  ys [T*k, H], y [T, H] of one type; weights fp32 [T, k]."""
    where = "bq_moe_combine"
    st = _on_stream(where, stream, ys, inv, weights, y)
    po, dt, t, h, ldo = _rows_of(where, "y", y)
    if t == 0:
        return y
    pi, k = _pairs(where, inv, t)
    px, _, _, _, ldx = _rows_of(where, "ys", ys, t * k, h, dt)
    pw = _dense(where, "weights", weights, (t, k), "f32")
    _check(_lib.bq_moe_combine(px, dt, t, h, ldx, pi, pw, k, int(bool(accumulate)), po, ldo, st), where)
    return y


def moe_combine_backward(dy, ys, inv, weights, dys, dweights, stream=None):
    """Gradients of moe_combine: dys[inv[t][j]] = weights[t][j] * dy[t] and
    dweights[t][j] = <dy[t], ys[inv[t][j]]>.  dys or dweights may be None (not
    computed; then weights, or ys, may be None too)."""
    where = "bq_moe_combine_backward"
    st = _on_stream(where, stream, dy, ys, inv, weights, dys, dweights)
    pg, dt, t, h, ldg = _rows_of(where, "dy", dy)
    if t == 0:
        return dys, dweights
    pi, k = _pairs(where, inv, t)
    px, ldx = None, 0
    if ys is not None:
        px, _, _, _, ldx = _rows_of(where, "ys", ys, t * k, h, dt)
    po, ldo = None, 0
    if dys is not None:
        po, _, _, _, ldo = _rows_of(where, "dys", dys, t * k, h, dt)
    pw = None if weights is None else _dense(where, "weights", weights, (t, k), "f32")
    pd = None if dweights is None else _dense(where, "dweights", dweights, (t, k), "f32")
    _check(_lib.bq_moe_combine_backward(pg, ldg, px, ldx, dt, t, h, pi, pw, k, po, ldo, pd, st), where)
    return dys, dweights


def quant_fp8_b128(x, q, scales, n_rows=None, stream=None):
    """Rows to FP8 e4m3, one fp32 scale per 128 values.  x [rows, k] fp32, fp16 or
    bf16 (k a multiple of 16); q [rows, k] float8_e4m3fn or uint8; scales fp32
    [rows, ceil(k/128)].  n_rows: optional int32 device tensor of one element, the
    number of rows to quantise (the others are left as they are)."""
    where = "bq_quant_fp8_b128"
    st = _on_stream(where, stream, x, q, scales, n_rows)
    px, dt, r, k, ldx = _rows_of(where, "x", x)
    pq = _dense(where, "q", q, (r, k), "fp8")
    ps = _dense(where, "scales", scales, (r, -(-k // 128)), "f32")
    pn = None if n_rows is None else _dense(where, "n_rows", n_rows.view(-1), (1,), "i32")
    _check(_lib.bq_quant_fp8_b128(px, dt, r, k, ldx, pn, pq, ps, st), where)
    return q, scales


def moe_dispatch_fp8_b128(x, inv, q, scales, stream=None):
    """moe_dispatch and quant_fp8_b128 in one pass: q [T*k, H] and scales
    [T*k, ceil(H/128)] in expert order."""
    where = "bq_moe_dispatch_fp8_b128"
    st = _on_stream(where, stream, x, inv, q, scales)
    px, dt, t, h, ldx = _rows_of(where, "x", x)
    if t == 0:
        return q, scales
    pi, k = _pairs(where, inv, t)
    pq = _dense(where, "q", q, (t * k, h), "fp8")
    ps = _dense(where, "scales", scales, (t * k, -(-h // 128)), "f32")
    _check(_lib.bq_moe_dispatch_fp8_b128(px, dt, t, h, ldx, pi, k, pq, ps, st), where)
    return q, scales


def _product(where, x, x_scales, w, w_scales, y, swiglu, grouped):
    wshape = w.shape
    if len(x.shape) != 2 or len(wshape) != (3 if grouped else 2):
        _refuse(2, where, f"x has shape {list(x.shape)}, w {list(wshape)}")
    m, k = x.shape
    n = wshape[-2]
    if max(m, k, *wshape) > 0x7fffffff:
        _refuse(2, where, f"x has shape {list(x.shape)}, w {list(wshape)}")
    kb, nb = (k + 127) // 128, (n + 127) // 128
    px = _dense(where, "x", x, (m, k), "fp8")
    pxs = _dense(where, "x_scales", x_scales, (m, kb), "f32")
    pw = _dense(where, "w", w, (wshape[0], n, k) if grouped else (n, k), "fp8")
    pws = _dense(where, "w_scales", w_scales, (wshape[0], nb, kb) if grouped else (nb, kb), "f32")
    py, dt, _, _, ldy = _rows_of(where, "y", y, m, n // 2 if swiglu else n)
    return px, pxs, m, pw, pws, n, k, 1 if swiglu else 0, py, dt, ldy


# bq_activation
ACT_NONE, ACT_SWIGLU, ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU, ACT_RELU2 = range(7)
ACT_BY_NAME = {"none": ACT_NONE, "swiglu": ACT_SWIGLU, "silu": ACT_SILU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH,
               "relu": ACT_RELU, "relu2": ACT_RELU2}


def _epilogue(where, swiglu, act, bias, bias_shape, residual, scale, dt, rows, cols):
    """bq_epilogue of a product's end, or None where it changes nothing."""
    if act is not None and act not in ACT_BY_NAME:
        _refuse(2, where, f"unknown activation {act!r}")
    code = ACT_SWIGLU if swiglu else ACT_NONE if act is None else ACT_BY_NAME[act]
    if bias is None and residual is None and scale == 1.0 and code <= ACT_SWIGLU:
        return None
    pb = None if bias is None else _dense(where, "bias", bias, bias_shape, "f32")
    pr, ldr = None, 0
    if residual is not None:
        pr, _, _, _, ldr = _rows_of(where, "residual", residual, rows, cols, dt)
    return _EPILOGUE.pack(code, scale, pb or 0, pr or 0, ldr)


def _gated(where, swiglu, act):
    if swiglu and act not in (None, "swiglu"):
        _refuse(2, where, f"swiglu and act={act!r} exclude each other")
    return swiglu or act == "swiglu"


def mm_fp8_b128(x, x_scales, w, w_scales, y, swiglu: bool = False, stream=None, *, act: str | None = None, bias=None,
                residual=None, scale: float = 1.0):
    """y = x w^T of FP8 rows x [m, k] (quant_fp8_b128) and an FP8 weight w [n, k] with
    one scale per 128 x 128 block; y [m, n] fp32, fp16 or bf16.  swiglu (or act="swiglu"):
    w holds n/2 gate rows and n/2 up rows, y [m, n/2] = silu(gate) * up.  With any of act
    (silu, gelu, gelu_tanh, relu, relu2), bias (fp32 [n]), scale and residual (rows like
    y's; it may be y): y = scale * act(x w^T + bias) + residual."""
    where = "bq_mm_fp8_b128"
    st = _on_stream(where, stream, x, x_scales, w, w_scales, y, bias, residual)
    swiglu = _gated(where, swiglu, act)
    px, pxs, m, pw, pws, n, k, sw, py, dt, ldy = _product(where, x, x_scales, w, w_scales, y, swiglu, False)
    epi = _epilogue(where, swiglu, act, bias, (n,), residual, scale, dt, m, y.shape[1])
    if epi is None:
        _check(_lib.bq_mm_fp8_b128(px, pxs, m, pw, pws, n, k, sw, py, dt, ldy, st), where)
    else:
        _check(_lib.bq_mm_fp8_b128_epilogue(px, pxs, m, pw, pws, n, k, epi, py, dt, ldy, st), where)
    return y


def moe_mm_fp8_b128(x, x_scales, offsets, w, w_scales, y, swiglu: bool = False, stream=None, *, act: str | None = None,
                    bias=None, residual=None, scale: float = 1.0):
    """mm_fp8_b128 over rows sorted by expert: rows offsets[e] .. offsets[e + 1] of x
    take w[e] (and bias[e]).  w [E, n, k], w_scales [E, ceil(n/128), ceil(k/128)], bias
    fp32 [E, n], offsets int32 [E + 1] from moe_permute.  Rows of y behind offsets[E]
    are left as they are."""
    where = "bq_moe_mm_fp8_b128"
    st = _on_stream(where, stream, x, x_scales, offsets, w, w_scales, y, bias, residual)
    swiglu = _gated(where, swiglu, act)
    px, pxs, m, pw, pws, n, k, sw, py, dt, ldy = _product(where, x, x_scales, w, w_scales, y, swiglu, True)
    e = w.shape[0]
    po = _dense(where, "offsets", offsets, (e + 1,), "i32")
    epi = _epilogue(where, swiglu, act, bias, (e, n), residual, scale, dt, m, y.shape[1])
    if epi is None:
        _check(_lib.bq_moe_mm_fp8_b128(px, pxs, m, po, e, pw, pws, n, k, sw, py, dt, ldy, st), where)
    else:
        _check(_lib.bq_moe_mm_fp8_b128_epilogue(px, pxs, m, po, e, pw, pws, n, k, epi, py, dt, ldy, st),
               where)
    return y


# ---------------------------------------------------------------- block to block
GATE_NONE, GATE_TOKEN, GATE_CHANNEL, GATE_FULL = 0, 1, 2, 3


def _vector(where: str, what: str, t, n: int):
    """(pointer, bq_dtype) of a contiguous vector of n elements of a row type."""
    if _DT is None:
        _load_torch()
    dt = _DT.get(t.dtype)
    if dt is None:
        _refuse(4, where, f"{what} has type {t.dtype}")
    if t.shape != (n,) or not t.is_contiguous():
        _refuse(2, where, f"{what} has shape {list(t.shape)} and strides {tuple(t.stride())}, expected contiguous [{n}]")
    return t.data_ptr(), dt


def _workspace(where: str, t):
    """(pointer, bytes) of a workspace, or (None, 0).  A tensor that holds fewer bytes than it has elements (an expanded
    one) would be written past its end."""
    if t is None:
        return None, 0
    if not t.is_contiguous():
        _refuse(3, where, f"the workspace has shape {list(t.shape)} and strides {tuple(t.stride())}, expected a contiguous one")
    return t.data_ptr(), t.numel() * t.element_size()


def _gate(where: str, gate, t: int, h: int):
    """(kind, pointer, bq_dtype, row stride) of a gate [T, 1], [H] or [T, H]."""
    if gate is None:
        return GATE_NONE, None, DT_F32, 0
    shape = gate.shape
    if len(shape) == 1:
        return (GATE_CHANNEL, *_vector(where, "gate", gate, h), 0)
    if shape == (t, 1):
        return (GATE_TOKEN, *_vector(where, "gate", gate.view(-1) if gate.is_contiguous() else gate, t), 0)
    p, dt, _, _, ld = _rows_of(where, "gate", gate, t, h)
    return GATE_FULL, p, dt, ld


def _norm_desc(where, t, h, dy, dh, dx, gain, post_gain, gate, gate_sigmoid, scale, residual_scale, eps):
    pg, gdt = (None, None) if gain is None else _vector(where, "gain", gain, h)
    pp, pdt = (None, gdt) if post_gain is None else _vector(where, "post_gain", post_gain, h)
    if gdt is not None and pdt != gdt:
        _refuse(4, where, f"gain has type {gain.dtype}, post_gain {post_gain.dtype}")
    kind, pgate, gate_dt, ldgate = _gate(where, gate, t, h)
    return kind, gate_dt, _RESIDUAL_NORM_DESC.pack(t, h, dy, dh, dx, DT_F32 if pdt is None else pdt, gate_dt, kind,
                                                   int(bool(gate_sigmoid)), scale, residual_scale, eps, pg or 0, pp or 0,
                                                   pgate or 0, ldgate)


def residual_norm(y, h, h_out, x=None, gain=None, post_gain=None, gate=None, gate_sigmoid: bool = False,
                  scale: float = 1.0, residual_scale: float = 1.0, eps: float = 1e-6, stream=None):
    """A block's output y into the residual stream, and the stream normalised for the
    next block: h_out = residual_scale * h + scale * g * (post_gain * n(y), or y),
    x = gain * n(h_out), n(v) = v / sqrt(mean(v^2) + eps) per row.  g: gate [T, 1],
    [H] or [T, H], or its sigmoid.  y, h, x [T, H] of any row type each (h_out of h's;
    it may be h); gains [H] of one type.  x None: only h_out."""
    where = "bq_residual_norm"
    st = _on_stream(where, stream, y, h, h_out, x, gain, post_gain, gate)
    py, dy, t, n, ldy = _rows_of(where, "y", y)
    ph, dh, _, _, ldh = _rows_of(where, "h", h, t, n)
    po, _, _, _, ldo = _rows_of(where, "h_out", h_out, t, n, dh)
    px, dx, ldx = None, dh, 0
    if x is not None:
        px, dx, _, _, ldx = _rows_of(where, "x", x, t, n)
    _, _, desc = _norm_desc(where, t, n, dy, dh, dx, gain, post_gain, gate, gate_sigmoid, scale, residual_scale, eps)
    _check(_lib.bq_residual_norm(desc, py, ldy, ph, ldh, po, ldo, px, ldx, st), where)
    return h_out, x


def residual_norm_backward_workspace_bytes(t: int, h: int) -> int:
    return int(_lib.bq_residual_norm_backward_workspace_bytes(t, h))


def residual_norm_backward(y, h_out, dh_out, dx, dy, dh, gain=None, post_gain=None, gate=None,
                           gate_sigmoid: bool = False, scale: float = 1.0, residual_scale: float = 1.0,
                           eps: float = 1e-6, dgain=None, dpost_gain=None, dgate=None, workspace=None, stream=None):
    """Gradients of residual_norm from those of h_out and x (dh_out or dx may be None):
    dy, dh (may be dh_out), and where given dgain, dpost_gain (fp32 [H]) and dgate (the
    gate's shape; fp32, or the gate's type for a gate [T, H]).  The sums over rows need
    a workspace of residual_norm_backward_workspace_bytes(T, H) bytes (uint8)."""
    where = "bq_residual_norm_backward"
    st = _on_stream(where, stream, y, h_out, dh_out, dx, dy, dh, gain, post_gain, gate, dgain, dpost_gain, dgate,
                    workspace)
    py, ty, t, n, ldy = _rows_of(where, "y", y)
    pd, _, _, _, ldd = _rows_of(where, "dy", dy, t, n, ty)
    pg, th, _, _, ldg = _rows_of(where, "dh", dh, t, n)
    ph, ldh, po, ldo, px, ldx, tx = None, 0, None, 0, None, 0, th
    if h_out is not None:
        ph, _, _, _, ldh = _rows_of(where, "h_out", h_out, t, n, th)
    if dh_out is not None:
        po, _, _, _, ldo = _rows_of(where, "dh_out", dh_out, t, n, th)
    if dx is not None:
        px, tx, _, _, ldx = _rows_of(where, "dx", dx, t, n)
    kind, gate_dt, desc = _norm_desc(where, t, n, ty, th, tx, gain, post_gain, gate, gate_sigmoid, scale, residual_scale, eps)
    sums = [None if s is None else _dense(where, what, s, (n,), "f32")
            for what, s in (("dgain", dgain), ("dpost_gain", dpost_gain))]
    pgate, ldgate = None, 0
    if dgate is not None:
        if gate is None or dgate.shape != gate.shape:
            _refuse(2, where, f"dgate has shape {list(dgate.shape)}, the gate "
                              f"{None if gate is None else list(gate.shape)}")
        if kind == GATE_FULL:
            pgate, _, _, _, ldgate = _rows_of(where, "dgate", dgate, t, n, gate_dt)
        else:
            pgate = _dense(where, "dgate", dgate, gate.shape, "f32")
    pw, nw = _workspace(where, workspace)
    _check(_lib.bq_residual_norm_backward(desc, py, ldy, ph, ldh, po, ldo, px, ldx, pd, ldd, pg, ldg,
                                          *sums, pgate, ldgate, pw, nw, st), where)
    return dy, dh


# ---------------------------------------------------------------- router training
def _router(where, logits, ids, seq_offsets):
    if len(logits.shape) != 2:
        _refuse(2, where, f"logits has shape {list(logits.shape)}, expected [T, E]")
    t, e = logits.shape
    if len(ids.shape) != 2 or t > 0x7fffffff:
        _refuse(2, where, f"ids has shape {list(ids.shape)}, logits {list(logits.shape)}")
    k = ids.shape[1]
    pl = _dense(where, "logits", logits, (t, e), "f32")
    pi = _dense(where, "ids", ids, (t, k), "i32")
    ps, s = None, 1
    if seq_offsets is not None:
        s = seq_offsets.numel() - 1
        ps = _dense(where, "seq_offsets", seq_offsets, (s + 1,), "i32")
    return pl, pi, t, e, k, ps, s


def moe_balance_workspace_bytes(t: int, e: int, sequences: int = 1) -> int:
    return int(_lib.bq_moe_balance_workspace_bytes(t, e, sequences))


def moe_balance_loss(logits, ids, counts, probs, losses, workspace, bias=None, scoring: int = SCORE_SOFTMAX,
                     seq_offsets=None, stream=None):
    """Balance statistics of a router's logits (fp32 [T, E]) and its ids (int32 [T, k]), over
    all rows or per sequence (seq_offsets int32 [S + 1]): counts int32 and probs fp32 [S, E]
    (S = 1 without offsets), losses fp32 [2]: the balance loss (1 for an even load) and the
    z-loss.  bias: of the softmax rule.  workspace: moe_balance_workspace_bytes(T, E, S)."""
    where = "bq_moe_balance_loss"
    st = _on_stream(where, stream, logits, ids, counts, probs, losses, workspace, bias, seq_offsets)
    pl, pi, t, e, k, ps, s = _router(where, logits, ids, seq_offsets)
    pb = None if bias is None else _dense(where, "bias", bias, (e,), "f32")
    pc = _dense(where, "counts", counts, (s, e), "i32")
    pp = _dense(where, "probs", probs, (s, e), "f32")
    po = _dense(where, "losses", losses, (2,), "f32")
    _check(_lib.bq_moe_balance_loss(pl, pb, t, e, pi, k, scoring, ps, s, pc, pp, po, *_workspace(where, workspace), st),
           where)
    return counts, probs, losses


def moe_route_backward_workspace_bytes(t: int, e: int) -> int:
    return int(_lib.bq_moe_route_backward_workspace_bytes(t, e))


def moe_route_backward(logits, ids, dweights, dlogits, bias=None, scoring: int = SCORE_SOFTMAX, scale: float = 1.0,
                       counts=None, dlosses=None, seq_offsets=None, dbias=None, workspace=None, stream=None):
    """Gradient of the router's weights (dweights fp32 [T, k], or None) and of the two losses of
    moe_balance_loss (dlosses fp32 [2] with its counts, or None) with respect to the logits:
    dlogits [T, E] of any row type; rows in no sequence stay as they were.  dbias fp32 [E] (softmax
    rule) needs a workspace of moe_route_backward_workspace_bytes(T, E) bytes."""
    where = "bq_moe_route_backward"
    st = _on_stream(where, stream, logits, ids, dweights, dlogits, bias, counts, dlosses, seq_offsets, dbias, workspace)
    pl, pi, t, e, k, ps, s = _router(where, logits, ids, seq_offsets)
    if not dlogits.is_contiguous():
        _refuse(2, where, f"dlogits has strides {tuple(dlogits.stride())}")
    po, dt, _, _, _ = _rows_of(where, "dlogits", dlogits, t, e)
    vectors = [None if v is None else _dense(where, what, v, shape, kind)
               for what, v, shape, kind in (("bias", bias, (e,), "f32"), ("dweights", dweights, (t, k), "f32"),
                                            ("counts", counts, (s, e), "i32"), ("dlosses", dlosses, (2,), "f32"),
                                            ("dbias", dbias, (e,), "f32"))]
    pb, pw, pc, pd, pdb = vectors
    ws, nw = _workspace(where, workspace)
    _check(_lib.bq_moe_route_backward(pl, pb, t, e, pi, k, scoring, scale, pw, pc, pd, ps, s, po, dt, pdb, ws, nw, st),
           where)
    return dlogits
