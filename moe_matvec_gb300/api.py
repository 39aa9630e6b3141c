"""Python binding of the C-ABI library libqmv.so (see include/qmv.h).

Argument marshalling only (ctypes; for the norm, cache, attention and page
selection calls of a decode layer a native module, csrc/binding.cpp, and for
rotation, adapters, expert selection and log probabilities another,
csrc/binding_step.cpp): every computation runs in the library's CUDA kernels.  Tensors are torch CUDA tensors (PyTorch supplies device memory and
the current stream); results are returned as new tensors unless `out` is
given.  There is no CPU fallback: importing this module without a buildable
library raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import build as _build

Q8_0, Q4_K, IQ4_XS, Q5_K, Q6_K, Q8_G64, Q8_G128, F16, F32 = 0, 1, 2, 3, 4, 5, 6, 7, 8
FORMATS = {"Q8_0": Q8_0, "Q4_K": Q4_K, "IQ4_XS": IQ4_XS, "Q5_K": Q5_K, "Q6_K": Q6_K, "Q8_G64": Q8_G64,
           "Q8_G128": Q8_G128, "F16": F16, "F32": F32}
GROUP_WEIGHTS = {Q8_0: 256, Q4_K: 256, IQ4_XS: 512, Q5_K: 256, Q6_K: 256, Q8_G64: 512, Q8_G128: 1024,
                 F16: 32, F32: 32}
BYTES_PER_WEIGHT = {Q8_0: 272 / 256, Q4_K: 144 / 256, IQ4_XS: 272 / 512, Q5_K: 176 / 256, Q6_K: 208 / 256,
                    Q8_G64: 528 / 512, Q8_G128: 1040 / 1024, F16: 2.0, F32: 4.0}
MAX_TOKENS = 64
MAX_TOPK = 8

DEVERR_EXPERT_RANGE = 0x1
DEVERR_EXPERT_DUP = 0x2
DEVERR_TIMEOUT = 0x4
DEVERR_RANGE = 0x8
DEVERR_PAGE = 0x10
DEVERR_BATCH = 0x20
DEVERR_ADAPTER = 0x40
DEVERR_TOKEN = 0x80


class QmvError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} ({code})")
        self.code = code


class MoeExperts(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int32), ("hidden", ctypes.c_int32), ("ffn", ctypes.c_int32),
                ("fmt_gate_up", ctypes.c_int32), ("fmt_down", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("w_gate_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p)]


class KvCache(ctypes.Structure):
    _fields_ = [("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("pages", ctypes.c_void_p), ("bounds", ctypes.c_void_p)]


class KvBatch(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("starts", ctypes.c_void_p),
                ("n_seq", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("n_tok", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Rope(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("n_axes", ctypes.c_int32), ("scale", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("freq", ctypes.c_void_p), ("axis", ctypes.c_void_p)]


class Lora(ctypes.Structure):
    _fields_ = [("n_adapters", ctypes.c_int32), ("rank", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("ranks", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_i64, _vp, _int, _sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_SIGS = {
    "qmv_row_bytes": (_i64, [_int, _i64]),
    "qmv_quantize_weights": (_int, [_int, _vp, _i64, _i64, _vp, _vp]),
    "qmv_quantize_act": (_int, [_vp, _i64, _int, _vp, _vp, _vp, _vp]),
    "qmv_run": (_int, [_int, _vp, _vp, _vp, _i64, _i64, _int, _vp]),
    "qmv_run_q8": (_int, [_int, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _int, _vp]),
    "qmv_splitk_choose": (_int, [_int, _i64, _i64, _int]),
    "qmv_splitk_workspace_bytes": (_sz, [_i64, _int, _int]),
    "qmv_act_q8_bytes": (_sz, [_i64, _int]),
    "qmv_splitk_run": (_int, [_int, _vp, _vp, _vp, _i64, _i64, _int, _int, _vp, _sz, _vp]),
    "qmv_splitk_run_static": (_int, [_int, _vp, _vp, _vp, _i64, _i64, _int, _int, _vp]),
    "moe_qmv_workspace_bytes": (_sz, [ctypes.POINTER(MoeExperts), _int, _int]),
    "moe_qmv_workspace_offsets": (_int, [ctypes.POINTER(MoeExperts), _int, _int, ctypes.POINTER(_sz * 5)]),
    "moe_qmv_run": (_int, [ctypes.POINTER(MoeExperts), _vp, _vp, _vp, _vp, _int, _int, _vp, _sz, _vp]),
    "moe_qmv_prefill_workspace_bytes": (_sz, [ctypes.POINTER(MoeExperts), _int, _int]),
    "moe_qmv_prefill_workspace_offsets": (_int, [ctypes.POINTER(MoeExperts), _int, _int, ctypes.POINTER(_sz * 5)]),
    "moe_qmv_prefill_run": (_int, [ctypes.POINTER(MoeExperts), _vp, _vp, _vp, _vp, _int, _int, _vp, _sz, _vp]),
    "moe_route_run": (_int, [_int, _vp, _vp, _int, _i64, _int, _int, _int, _vp, _vp, _vp, _vp]),
    "qmv_run_residual": (_int, [_int, _vp, _vp, _vp, _vp, _i64, _i64, _int, _int, _vp, _sz, _vp]),
    "qmv_run_siblings": (_int, [_int, _vp, _vp, _vp, _vp, _vp, _i64, _int, _vp, _sz, _vp]),
    "qmv_rms_norm": (_int, [_int, _vp, _i64, _vp, _vp, ctypes.c_float, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "qmv_dequantize_act": (_int, [_int, _vp, _vp, _i64, _i64, _vp, _vp]),
    "qmv_kv_page_bytes": (_i64, [_int, _int]),
    "qmv_kv_bounds_bytes": (_i64, [_int]),
    "qmv_kv_append": (_int, [ctypes.POINTER(KvCache), ctypes.POINTER(KvBatch), _int, _vp, _i64, _vp, _i64, _vp]),
    "qmv_kv_read": (_int, [ctypes.POINTER(KvCache), ctypes.POINTER(KvBatch), _int, _vp, _vp, _vp]),
    "qmv_kv_attend_workspace_bytes": (_sz, [ctypes.POINTER(KvCache), _int, _int, _int]),
    "qmv_kv_attend": (_int, [ctypes.POINTER(KvCache), ctypes.POINTER(KvBatch), _int, _vp, _i64, _vp, _int,
                             ctypes.c_float, _int, _int, _vp, _int, _vp, _sz, _vp]),
    "qmv_kv_select_workspace_bytes": (_sz, [ctypes.POINTER(KvCache), ctypes.POINTER(KvBatch)]),
    "qmv_kv_select": (_int, [ctypes.POINTER(KvCache), ctypes.POINTER(KvBatch), _int, _vp, _i64, _int, _vp, _int,
                             _vp, _sz, _vp]),
    "qmv_norm_rope": (_int, [ctypes.POINTER(Rope), _int, _vp, _i64, _vp, _i64, _int, _vp, _vp, _i64, _vp, _i64, _int,
                             _vp, ctypes.c_float, _vp, _vp, _vp, _int, _int, _vp]),
    "qmv_lora_workspace_bytes": (_sz, [ctypes.POINTER(Lora), _i64, _int]),
    "qmv_lora_run": (_int, [ctypes.POINTER(Lora), _vp, _vp, _vp, _vp, _i64, _i64, _int, _vp, _sz, _vp]),
    "moe_route_select": (_int, [_int, _vp, _i64, _vp, _int, _int, _int, _int, _int, _int, _int, _int, ctypes.c_float,
                                _vp, _vp, _vp]),
    "qmv_logprobs": (_int, [_int, _vp, _i64, _i64, _i64, ctypes.c_float, _vp, _int, _vp, _vp, _vp, _int, _vp, _vp,
                            _vp]),
    "qmv_get_device_error": (_int, [_vp, ctypes.POINTER(_int)]),
    "qmv_debug_shrink_outputs": (_int, [_i64]),
    "qmv_wait_probe": (_int, [ctypes.c_longlong, _vp, _vp]),
    "qmv_tc_probe": (_int, [_vp, _vp, _int, _vp, _vp]),
    "qmv_measure_pipes_scratch_bytes": (_sz, []),
    "qmv_measure_pipes": (_int, [ctypes.POINTER(ctypes.c_double), _int, _vp, _sz, _vp]),
    "qmv_check_rounding": (_int, [_vp, _vp]),
    "qmv_strerror": (ctypes.c_char_p, [_int]),
}

_lib = None
_native = None  # the native module, driving _lib (None until a call needs it)
_step = None    # the second one, likewise
_NATIVE_CALLS = ("qmv_rms_norm", "qmv_dequantize_act", "qmv_kv_append", "qmv_kv_read", "qmv_kv_attend",
                 "qmv_kv_attend_workspace_bytes", "qmv_kv_select", "qmv_kv_select_workspace_bytes")
_STEP_CALLS = ("qmv_norm_rope", "qmv_lora_run", "qmv_lora_workspace_bytes", "moe_route_select", "qmv_logprobs")


def _bind(module, calls):
    """Point a native module at the active library."""
    module.bind(QmvError, *[ctypes.cast(getattr(_lib, n), ctypes.c_void_p).value for n in calls])


def _activate(lib):
    """Make `lib` the library that every call goes to."""
    global _lib
    _lib = lib
    if _native is not None:
        _bind(_native, _NATIVE_CALLS)
    if _step is not None:
        _bind(_step, _STEP_CALLS)
    return lib


def _open(path: str):
    if not os.path.exists(path):
        raise ImportError(f"library not found at {path}")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name, None)
        if fn is None:
            continue
        fn.restype = res
        fn.argtypes = args
    return lib


def load(path: str | None = None):
    """Load (building first if needed) libqmv.so and declare its signatures."""
    if _lib is not None:
        return _lib
    return _activate(_open(path or _build.build()))


_debug_lib = None


def load_debug():
    """The QMV_DEBUG build of the library (libqmv_debug.so: every kernel access
    range-checked in software, see qmv_debug_shrink_outputs in qmv.h), built if
    needed.  It is not made the current library: run calls through it with
    `using(load_debug())`."""
    global _debug_lib
    if _debug_lib is None:
        _debug_lib = _open(_build.build(debug=True))
    return _debug_lib


@contextlib.contextmanager
def using(lib):
    """Within the block, every call of this module goes to `lib` (a library
    from load() or load_debug())."""
    prev = load()
    _activate(lib)
    try:
        yield lib
    finally:
        _activate(prev)


def debug_shrink_outputs(n: int) -> None:
    """Debug library only (inside `using(load_debug())`): later calls hand the
    range checks their result buffers' extents n elements short (0 restores)."""
    _check(load().qmv_debug_shrink_outputs(int(n)), "qmv_debug_shrink_outputs")


def strerror(code: int) -> str:
    return load().qmv_strerror(int(code)).decode()


def _check(rc: int, what: str):
    if rc != 0:
        raise QmvError(rc, what)


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def row_bytes(fmt: int, K: int) -> int:
    rb = load().qmv_row_bytes(int(fmt), int(K))
    _check(rb if rb < 0 else 0, "qmv_row_bytes")
    return int(rb)


def quantize_weights(fmt: int, w: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 weights [M][K] -> rows of format fmt, uint8 [M][row_bytes] (F16 / F32: the values
    converted, binary16 rounded to nearest even)."""
    M, K = w.shape
    rb = row_bytes(fmt, K)
    if out is None:
        out = torch.empty((M, rb), dtype=torch.uint8, device=w.device)
    _check(load().qmv_quantize_weights(int(fmt), _ptr(w), M, K, _ptr(out), _stream(stream)), "qmv_quantize_weights")
    return out


def quantize_act(x: torch.Tensor, stream=None):
    """Activation rule on x fp32 [n][K] -> (q int8 [n][K], d fp32 [n][K/32], s int32 [n][K/32]) in the
    library's Q8 activation layout (codes of each 256-element group halves first, see qmv.h)."""
    n, K = x.shape
    q = torch.empty((n, K), dtype=torch.int8, device=x.device)
    d = torch.empty((n, K // 32), dtype=torch.float32, device=x.device)
    s = torch.empty((n, K // 32), dtype=torch.int32, device=x.device)
    _check(load().qmv_quantize_act(_ptr(x), K, n, _ptr(q), _ptr(d), _ptr(s), _stream(stream)), "qmv_quantize_act")
    return q, d, s


def run(fmt: int, W: torch.Tensor, x: torch.Tensor, M: int, K: int, out: torch.Tensor | None = None,
        stream=None) -> torch.Tensor:
    """y [n][M] = What x Xhat (quantized matvec; F16 / F32 rows: Xhat = x), x fp32 [n][K]."""
    n = x.shape[0]
    if out is None:
        out = torch.empty((n, M), dtype=torch.float32, device=x.device)
    _check(load().qmv_run(int(fmt), _ptr(W), _ptr(x), _ptr(out), M, K, n, _stream(stream)), "qmv_run")
    return out


def run_q8(fmt: int, W: torch.Tensor, xq: torch.Tensor, xd: torch.Tensor, xs: torch.Tensor, M: int, K: int,
           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Matvec with activations already quantized by quantize_act (quantized formats only)."""
    n = xq.shape[0]
    if out is None:
        out = torch.empty((n, M), dtype=torch.float32, device=xq.device)
    _check(load().qmv_run_q8(int(fmt), _ptr(W), _ptr(xq), _ptr(xd), _ptr(xs), _ptr(out), M, K, n, _stream(stream)),
           "qmv_run_q8")
    return out


def splitk_choose(fmt: int, M: int, K: int, n_tok: int) -> int:
    s = load().qmv_splitk_choose(int(fmt), M, K, n_tok)
    _check(s if s < 0 else 0, "qmv_splitk_choose")
    return int(s)


def splitk_workspace_bytes(M: int, n_tok: int, n_split: int) -> int:
    return int(load().qmv_splitk_workspace_bytes(M, n_tok, n_split))


def act_q8_bytes(K: int, n_tok: int) -> int:
    return int(load().qmv_act_q8_bytes(K, n_tok))


def splitk_workspace_fast_bytes(M: int, K: int, n_tok: int, n_split: int) -> int:
    """Workspace that lets qmv_splitk_run quantize the activations once."""
    part = splitk_workspace_bytes(M, n_tok, n_split) if n_split > 1 else 0
    return ((part + 255) // 256) * 256 + act_q8_bytes(K, n_tok)


def splitk_run(fmt: int, W: torch.Tensor, x: torch.Tensor, M: int, K: int, n_split: int = 0,
               ws: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Split-K matvec; n_split = 0 picks the split from the shape.  Without a
    given workspace, one large enough for pre-quantized activations is made."""
    n = x.shape[0]
    if n_split == 0:
        n_split = splitk_choose(fmt, M, K, n)
    if out is None:
        out = torch.empty((n, M), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = torch.empty(max(16, splitk_workspace_fast_bytes(M, K, n, n_split)), dtype=torch.uint8, device=x.device)
    wsb = ws.numel() * ws.element_size() if ws is not None else 0
    _check(load().qmv_splitk_run(int(fmt), _ptr(W), _ptr(x), _ptr(out), M, K, n, n_split, _ptr(ws), wsb,
                                 _stream(stream)), "qmv_splitk_run")
    return out


def run_residual(fmt: int, W: torch.Tensor, x: torch.Tensor, r: torch.Tensor, M: int, K: int,
                 out: torch.Tensor | None = None, n_split: int = 0, ws: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """y = What Xhat + r (r fp32 [n][M]; out may be r for y += What Xhat)."""
    n = x.shape[0]
    if n_split == 0:
        n_split = splitk_choose(fmt, M, K, n)
    if out is None:
        out = torch.empty((n, M), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = torch.empty(max(16, splitk_workspace_fast_bytes(M, K, n, n_split)), dtype=torch.uint8, device=x.device)
    _check(load().qmv_run_residual(int(fmt), _ptr(W), _ptr(x), _ptr(r), _ptr(out), M, K, n, n_split, _ptr(ws),
                                   ws.numel(), _stream(stream)), "qmv_run_residual")
    return out


def run_siblings(mats, x: torch.Tensor, K: int, outs=None, ws: torch.Tensor | None = None, stream=None):
    """Sibling matvecs sharing x: mats is a list of (fmt, W, M); returns the
    list of y_i fp32 [n][M_i]."""
    n = x.shape[0]
    c = len(mats)
    if outs is None:
        outs = [torch.empty((n, M), dtype=torch.float32, device=x.device) for _, _, M in mats]
    if ws is None:
        ws = torch.empty(max(16, act_q8_bytes(K, n)), dtype=torch.uint8, device=x.device)
    fm = (ctypes.c_int * c)(*[int(f) for f, _, _ in mats])
    Wp = (ctypes.c_void_p * c)(*[W.data_ptr() for _, W, _ in mats])
    Mp = (ctypes.c_int64 * c)(*[int(M) for _, _, M in mats])
    yp = (ctypes.c_void_p * c)(*[o.data_ptr() for o in outs])
    _check(load().qmv_run_siblings(c, fm, Wp, Mp, yp, _ptr(x), K, n, _ptr(ws), ws.numel(), _stream(stream)),
           "qmv_run_siblings")
    return outs


STATIC_SCRATCH_BYTES = 8 << 20


def splitk_run_static(fmt: int, W: torch.Tensor, x: torch.Tensor, M: int, K: int, n_split: int = 0,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Split-K matvec for callers that cannot allocate: the partial sums use
    the library's static device array (see qmv_splitk_run_static)."""
    n = x.shape[0]
    if out is None:
        out = torch.empty((n, M), dtype=torch.float32, device=x.device)
    _check(load().qmv_splitk_run_static(int(fmt), _ptr(W), _ptr(x), _ptr(out), M, K, n, n_split, _stream(stream)),
           "qmv_splitk_run_static")
    return out


def moe_experts(n_experts: int, hidden: int, ffn: int, fmt_gate_up: int, fmt_down: int, w_gate_up: torch.Tensor,
                w_down: torch.Tensor) -> MoeExperts:
    """The expert pool descriptor.  It holds references to the two weight
    tensors, so their device memory stays allocated as long as the descriptor
    lives (the C struct itself keeps only their addresses)."""
    e = MoeExperts(n_experts, hidden, ffn, fmt_gate_up, fmt_down, 0, _ptr(w_gate_up), _ptr(w_down))
    e._tensors = (w_gate_up, w_down)
    return e


def moe_workspace_bytes(e: MoeExperts, n_tok: int, top_k: int) -> int:
    return int(load().moe_qmv_workspace_bytes(ctypes.byref(e), n_tok, top_k))


def moe_workspace_offsets(e: MoeExperts, n_tok: int, top_k: int):
    arr = (_sz * 5)()
    _check(load().moe_qmv_workspace_offsets(ctypes.byref(e), n_tok, top_k, ctypes.byref(arr)),
           "moe_qmv_workspace_offsets")
    return list(arr)


def moe_run(e: MoeExperts, ids: torch.Tensor, gates: torch.Tensor, x: torch.Tensor, ws: torch.Tensor | None = None,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Expert-grouped MoE decode layer; ids int32 [n][top_k], gates fp32 [n][top_k], x fp32 [n][hidden]."""
    n, top_k = ids.shape
    if out is None:
        out = torch.empty((n, e.hidden), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = torch.empty(moe_workspace_bytes(e, n, top_k), dtype=torch.uint8, device=x.device)
    _check(load().moe_qmv_run(ctypes.byref(e), _ptr(ids), _ptr(gates), _ptr(x), _ptr(out), n, top_k, _ptr(ws),
                              ws.numel(), _stream(stream)), "moe_qmv_run")
    return out


MAX_PREFILL_TOKENS = 16384


def moe_prefill_workspace_bytes(e: MoeExperts, n_tok: int, top_k: int) -> int:
    return int(load().moe_qmv_prefill_workspace_bytes(ctypes.byref(e), n_tok, top_k))


def moe_prefill_workspace_offsets(e: MoeExperts, n_tok: int, top_k: int):
    arr = (_sz * 5)()
    _check(load().moe_qmv_prefill_workspace_offsets(ctypes.byref(e), n_tok, top_k, ctypes.byref(arr)),
           "moe_qmv_prefill_workspace_offsets")
    return list(arr)


def moe_prefill_run(e: MoeExperts, ids: torch.Tensor, gates: torch.Tensor, x: torch.Tensor,
                    ws: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The MoE layer for large batches on the tensor cores (moe_qmv_prefill_run);
    arguments as moe_run, n up to MAX_PREFILL_TOKENS."""
    n, top_k = ids.shape
    if out is None:
        out = torch.empty((n, e.hidden), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = torch.empty(moe_prefill_workspace_bytes(e, n, top_k), dtype=torch.uint8, device=x.device)
    _check(load().moe_qmv_prefill_run(ctypes.byref(e), _ptr(ids), _ptr(gates), _ptr(x), _ptr(out), n, top_k,
                                      _ptr(ws), ws.numel(), _stream(stream)), "moe_qmv_prefill_run")
    return out


GATING_SOFTMAX, GATING_SIGMOID = 0, 1


def route_run(fmt: int, Wr: torch.Tensor, x: torch.Tensor, n_experts: int, hidden: int, top_k: int,
              gating: int = GATING_SOFTMAX, logits: torch.Tensor | None = None, ids: torch.Tensor | None = None,
              gates: torch.Tensor | None = None, stream=None):
    """Router and top-k: logits fp32 [n][E] = What_r Xhat, then per token the
    top_k experts by logit (ids int32 [n][top_k]) and their gates normalised
    over the picked ones (fp32 [n][top_k]).  Returns (ids, gates, logits)."""
    n = x.shape[0]
    dev = x.device
    if logits is None:
        logits = torch.empty((n, n_experts), dtype=torch.float32, device=dev)
    if ids is None:
        ids = torch.empty((n, top_k), dtype=torch.int32, device=dev)
    if gates is None:
        gates = torch.empty((n, top_k), dtype=torch.float32, device=dev)
    _check(load().moe_route_run(int(fmt), _ptr(Wr), _ptr(x), int(n_experts), int(hidden), n, int(top_k),
                                int(gating), _ptr(logits), _ptr(ids), _ptr(gates), _stream(stream)),
           "moe_route_run")
    return ids, gates, logits


# ---------------------------------------------------------------------------
# The attention half of a decode layer
# ---------------------------------------------------------------------------
MAX_SEQS = 1024
MAX_BATCH_TOKENS = 65535
_WANT = {"float": 1, "q8": 2, "both": 3}


def _native_module(name: str, calls):
    load()
    loader = importlib.machinery.ExtensionFileLoader(name, _build.build_binding(name))
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader(name, loader))
    loader.exec_module(module)
    _bind(module, calls)
    return module


def _nat():
    """The native module, built and loaded by the first call that goes through it
    (the calls that go through ctypes need none of Python's and torch's headers)."""
    global _native
    if _native is None:
        _native = _native_module("_binding", _NATIVE_CALLS)
    return _native


def _on(stream):
    return None if stream is None else stream.cuda_stream


def rms_norm(x: torch.Tensor, w: torch.Tensor, eps: float = 1e-6, r: torch.Tensor | None = None, want: str = "float",
             y: torch.Tensor | None = None, q8=None, res: torch.Tensor | None = None, stream=None):
    """Root-mean-square norm with the residual's addition (qmv_rms_norm): s = x + r,
    y = s / sqrt(mean(s^2) + eps) * w per row.  x [n][K] (rows may be strided), r like x
    or None, w fp32 [K].  want: "float" (y in x's type), "q8" (y in the library's Q8
    activation layout, for run_q8) or "both".  Returns (y, (q, d, s), res), None for what
    was not asked for (res = s in x's type: only with r); y, q8 and res may be given as
    outputs, res also as r itself."""
    code = _WANT.get(want)
    if code is None:
        raise ValueError(f"want is 'float', 'q8' or 'both', got {want!r}")
    return _nat().rms_norm(x, w, eps, r, code, y, q8, res, _on(stream))


def dequantize_act(q: torch.Tensor, d: torch.Tensor, dtype: torch.dtype = torch.float32,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values [n][K] that Q8 activations (q, d of quantize_act or rms_norm) stand for."""
    return _nat().dequantize_act(q, d, dtype, out, _on(stream))


def kv_page_bytes(head_dim: int, page_tokens: int) -> int:
    n = load().qmv_kv_page_bytes(int(head_dim), int(page_tokens))
    _check(n if n < 0 else 0, "qmv_kv_page_bytes")
    return int(n)


def kv_bounds_bytes(head_dim: int) -> int:
    n = load().qmv_kv_bounds_bytes(int(head_dim))
    _check(n if n < 0 else 0, "qmv_kv_bounds_bytes")
    return int(n)


def _bytes(t: torch.Tensor | None, shape, what: str):
    if t is None:
        return None
    if t.dtype is not torch.uint8 or t.shape != shape:
        raise ValueError(f"{what}: torch.uint8 {shape} wanted, got {t.dtype} {tuple(t.shape)}")
    return _ptr(t)


def kv_cache(n_kv_heads: int, head_dim: int, page_tokens: int, n_pages: int, pages: torch.Tensor | None = None,
             bounds: torch.Tensor | bool | None = None, device=None) -> KvCache:
    """The descriptor of a paged 8-bit key / value cache (qmv_kv_cache).  pages uint8
    [n_pages][n_kv_heads][kv_page_bytes] and bounds uint8 [n_pages][n_kv_heads]
    [kv_bounds_bytes] are made where not given (bounds: only for True).  It holds
    references to both tensors (`.page_tensor`, `.bounds_tensor`)."""
    pb = kv_page_bytes(head_dim, page_tokens)
    if n_kv_heads < 1 or n_pages < 1:
        raise QmvError(-2, "kv_cache")
    if pages is None:
        pages = torch.empty((n_pages, n_kv_heads, pb), dtype=torch.uint8, device=device or "cuda")
    if bounds is True:
        bounds = torch.empty((n_pages, n_kv_heads, kv_bounds_bytes(head_dim)), dtype=torch.uint8, device=pages.device)
    elif bounds is False:
        bounds = None
    c = KvCache(n_kv_heads, head_dim, page_tokens, n_pages, _bytes(pages, (n_pages, n_kv_heads, pb), "pages"),
                _bytes(bounds, (n_pages, n_kv_heads, kv_bounds_bytes(head_dim)), "bounds"))
    c.page_tensor, c.bounds_tensor = pages, bounds
    return c


def kv_append(cache: KvCache, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
              starts: torch.Tensor | None = None, stream=None) -> None:
    """Write the last tokens of each sequence into the cache (qmv_kv_append).  k, v
    [n_tok][n_kv_heads][D] (tokens may be strided); table int32 [n_seq][max_pages], lens
    int32 [n_seq] counting these tokens, starts int32 [n_seq + 1] (None: one token per
    sequence)."""
    _nat().kv_append(ctypes.addressof(cache), k, v, table, lens, starts, _on(stream))


def kv_read(cache: KvCache, table: torch.Tensor, lens: torch.Tensor, starts: torch.Tensor | None = None,
            n_tok: int | None = None, dtype: torch.dtype = torch.float32, k: torch.Tensor | None = None,
            v: torch.Tensor | None = None, stream=None):
    """The last tokens of each sequence as values (qmv_kv_read): (k, v), each
    [n_tok][n_kv_heads][D].  n_tok is starts[-1] (a host number; None with starts None)."""
    return _nat().kv_read(ctypes.addressof(cache), table, lens, starts, n_tok, dtype, k, v, _on(stream))


def kv_attend_workspace_bytes(cache: KvCache, n_heads: int, n_tok: int, n_seq: int) -> int:
    return int(load().qmv_kv_attend_workspace_bytes(ctypes.byref(cache), int(n_heads), int(n_tok), int(n_seq)))


def kv_attend(cache: KvCache, q: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
              starts: torch.Tensor | None = None, scale: float | None = None, causal: bool = True, window: int = 0,
              pages: torch.Tensor | None = None, ws: torch.Tensor | None = None, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """Attention of the last tokens of each sequence over the cache (qmv_kv_attend).
    q [n_tok][n_heads][D] (tokens may be strided), scale 1 / sqrt(D) if None, pages int32
    [n_tok][n_kv_heads][n_sel] (kv_select's; n_sel 0 is refused) or None for all.
    Returns out like q."""
    return _nat().kv_attend(ctypes.addressof(cache), q, table, lens, starts, scale, causal, window, pages, ws, out,
                            _on(stream))


def kv_select_workspace_bytes(cache: KvCache, n_tok: int, max_pages: int) -> int:
    b = KvBatch(None, None, None, 1, max_pages, n_tok, 0)
    return int(load().qmv_kv_select_workspace_bytes(ctypes.byref(cache), ctypes.byref(b)))


def kv_select(cache: KvCache, q: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, n_sel: int,
              starts: torch.Tensor | None = None, ws: torch.Tensor | None = None, ids: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """The n_sel pages worth attending to for each token and kv head (qmv_kv_select): ids
    int32 [n_tok][n_kv_heads][n_sel], ascending, -1 after the last; for kv_attend's pages.
    The cache must have bounds."""
    return _nat().kv_select(ctypes.addressof(cache), q, table, lens, starts, n_sel, ws, ids, _on(stream))


# ---------------------------------------------------------------------------
# The rest of a decode step: rotation, adapters, expert selection, log
# probabilities
# ---------------------------------------------------------------------------
MAX_RANK = 128
MAX_TOP = 32
MAX_GIVEN = 64
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def _stp():
    """The second native module, as _nat."""
    global _step
    if _step is None:
        _step = _native_module("_binding_step", _STEP_CALLS)
    return _step


def _together(first: torch.Tensor, *rest) -> int:
    """The index + 1 of the device that all these tensors are on."""
    for t in rest:
        if t is not None and t.device != first.device:
            raise ValueError(f"tensors on {first.device} and {t.device}")
    return first.device.index + 1


def rope(head_dim: int, freq: torch.Tensor, axis: torch.Tensor | None = None, n_axes: int = 1,
         interleaved: bool = False, scale: float = 1.0) -> Rope:
    """How a model's heads turn (qmv_rope).  freq fp32 [R / 2]: radians a position of each
    pair of the first R of head_dim values (pair i: values i and i + R / 2, or 2i and 2i + 1 if
    interleaved); axis uint8 [R / 2]: which of a token's n_axes positions each pair goes by
    (None: the first); scale multiplies the turned values.  It holds references to both
    tensors."""
    if freq.dim() != 1 or freq.dtype is not torch.float32:
        raise ValueError(f"freq: torch.float32 [R / 2] wanted, got {freq.dtype} {tuple(freq.shape)}")
    if axis is not None and (axis.dtype is not torch.uint8 or axis.shape != freq.shape):
        raise ValueError(f"axis: torch.uint8 {tuple(freq.shape)} wanted, got {axis.dtype} {tuple(axis.shape)}")
    r = Rope(int(head_dim), 2 * freq.numel(), int(interleaved), int(n_axes), float(scale), 0, _ptr(freq), _ptr(axis))
    r.reserved = _together(freq, axis)
    r._tensors = (freq, axis)
    return r


def norm_rope(rope: Rope, q: torch.Tensor, k: torch.Tensor | None = None, q_w: torch.Tensor | None = None,
              k_w: torch.Tensor | None = None, eps: float = 1e-6, pos: torch.Tensor | None = None,
              lens: torch.Tensor | None = None, starts: torch.Tensor | None = None,
              q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Norm of each query and key head and its rotation (qmv_norm_rope).  q [n_tok][n_heads][D]
    and k [n_tok][n_kv_heads][D] (tokens may be strided), q_w and k_w fp32 [D] (None: no norm).
    Positions: pos int32 [n_tok][n_axes], or lens int32 [n_seq] and starts int32 [n_seq + 1] (None:
    one token per sequence) as for kv_append.  q_out and k_out may be strided, and q and k
    themselves; else they overlap neither these nor each other.  Returns (q_out, k_out)."""
    return _stp().norm_rope(ctypes.addressof(rope), q, k, q_w, k_w, eps, pos, lens, starts, q_out, k_out, _on(stream))


def lora(A: torch.Tensor, B: torch.Tensor, scales: torch.Tensor | None = None,
         ranks: torch.Tensor | None = None) -> Lora:
    """A pool of low-rank adapters of one projection (qmv_lora): A [n][rank][K] and B [n][M][rank]
    of one float type, scales fp32 [n] (None: 1), ranks int32 [n] (None: rank; how many of an
    adapter's rows of A and columns of B count).  It holds references to the tensors."""
    if A.dtype not in _DTYPES or A.dim() != 3 or B.dim() != 3 or B.dtype is not A.dtype or \
            (B.shape[0], B.shape[2]) != tuple(A.shape[:2]):
        raise ValueError(f"A [n][rank][K] and B [n][M][rank] of one float type wanted, got {A.dtype} "
                         f"{tuple(A.shape)} and {B.dtype} {tuple(B.shape)}")
    n, rank, K = A.shape
    for t, dt, what in ((scales, torch.float32, "scales"), (ranks, torch.int32, "ranks")):
        if t is not None and (t.dtype is not dt or t.shape != (n,)):
            raise ValueError(f"{what}: {dt} ({n},) wanted, got {t.dtype} {tuple(t.shape)}")
    d = Lora(n, rank, _DTYPES[A.dtype], 0, _ptr(A), _ptr(B), _ptr(ranks), _ptr(scales))
    d.reserved = _together(A, B, ranks, scales)
    d._tensors = (A, B, ranks, scales)
    d.K, d.M = K, B.shape[1]
    return d


def lora_workspace_bytes(lora: Lora, n_tok: int) -> int:
    return int(load().qmv_lora_workspace_bytes(ctypes.byref(lora), lora.K, int(n_tok)))


def lora_run(lora: Lora, ids: torch.Tensor, x: torch.Tensor, r: torch.Tensor, out: torch.Tensor | None = None,
             ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[t] = r[t] + scale_a B_a (A_a x[t]) with a = ids[t], none for a negative id (qmv_lora_run):
    adapters of many requests beside a shared projection whose result is r.  ids int32 [n_tok], x
    fp32 [n_tok][K], r fp32 [n_tok][M]; out may be r, else out and ws overlap nothing."""
    return _stp().lora_run(ctypes.addressof(lora), lora.K, lora.M, ids, x, r, out, ws, _on(stream))


def route_select(logits: torch.Tensor, top_k: int, gating: int = GATING_SOFTMAX, bias: torch.Tensor | None = None,
                 groups: int = 1, keep: int = 1, group_top: int = 2, renorm: bool = True, scale: float = 1.0,
                 ids: torch.Tensor | None = None, gates: torch.Tensor | None = None, stream=None):
    """Experts from router logits [n][E] (rows may be strided) (moe_route_select): scores by
    gating, bias fp32 [E] added for the choice alone, the `keep` of `groups` groups with the
    largest sum of their group_top best, top_k of those; gates are the picks' scores, over
    their sum if renorm, times scale.  Returns (ids int32 [n][top_k], gates fp32 [n][top_k]) for
    moe_run and moe_prefill_run."""
    return _stp().route_select(logits, top_k, gating, bias, groups, keep, group_top, renorm, scale, ids, gates,
                               _on(stream))


def logprobs(logits: torch.Tensor, tokens: torch.Tensor | None = None, n_top: int = 0, scale: float = 1.0,
             logp: torch.Tensor | None = None, lse: torch.Tensor | None = None, entropy: torch.Tensor | None = None,
             ids: torch.Tensor | None = None, top: torch.Tensor | None = None, stream=None):
    """Log probabilities under softmax(scale * logits) (qmv_logprobs).  logits [rows][V] (rows may
    be strided), tokens int32 [rows][n] or None.  Returns (logp fp32 [rows][n] of the tokens, lse
    and entropy fp32 [rows], ids int32 and top fp32 [rows][n_top]: the largest logits' tokens and
    log probabilities), None for what was not asked for; each may be given as an output."""
    return _stp().logprobs(logits, tokens, n_top, scale, logp, lse, entropy, ids, top, _on(stream))


def check_rounding(stream=None):
    """Mismatch counts (division, reciprocal) of the quantizer's branch-free
    arithmetic against IEEE round-to-nearest over every input of its range."""
    bad = torch.zeros(2, dtype=torch.int64, device="cuda")
    _check(load().qmv_check_rounding(_ptr(bad), _stream(stream)), "qmv_check_rounding")
    return [int(v) for v in bad.cpu()]


def tc_probe(A: torch.Tensor, B: torch.Tensor, stream=None) -> torch.Tensor:
    """A int8 [128][32], B int8 [N][32] -> A B^T fp32 [128][N] through the
    tcgen05 tensor cores (codes as f16, fp32 accumulator)."""
    N = B.shape[0]
    out = torch.empty((128, N), dtype=torch.float32, device=A.device)
    _check(load().qmv_tc_probe(_ptr(A), _ptr(B), N, _ptr(out), _stream(stream)), "qmv_tc_probe")
    return out


PIPE_NAMES = ("dp4a", "prmt", "ffma", "ffma2", "i2f", "mma_sync_s8_mac", "mma_sync_f16_mac",
              "tcgen05_f16_n256_mac", "tcgen05_f16_n64_mac", "tcgen05_f16_n32_mac")


def measure_pipes(stream=None) -> dict:
    """Measured per-SM per-clock rates (see qmv_measure_pipes), by name."""
    L = load()
    scratch = torch.empty(int(L.qmv_measure_pipes_scratch_bytes()), dtype=torch.uint8, device="cuda")
    arr = (ctypes.c_double * len(PIPE_NAMES))()
    n = L.qmv_measure_pipes(arr, len(PIPE_NAMES), _ptr(scratch), scratch.numel(), _stream(stream))
    _check(n if n < 0 else 0, "qmv_measure_pipes")
    return {PIPE_NAMES[i]: float(arr[i]) for i in range(n)}


def wait_probe(limit_cycles: int, stream=None) -> int:
    """Runs the kernels' bounded mbarrier wait with `limit_cycles` as its limit
    on a barrier that never completes (qmv_wait_probe); returns the SM cycles
    the wait lasted before it gave up.  Sets QMV_DEVERR_TIMEOUT."""
    cyc = torch.zeros(1, dtype=torch.int64, device="cuda")
    _check(load().qmv_wait_probe(int(limit_cycles), _ptr(cyc), _stream(stream)), "qmv_wait_probe")
    return int(cyc.item())


def get_device_error(stream=None) -> int:
    v = _int(0)
    _check(load().qmv_get_device_error(_stream(stream), ctypes.byref(v)), "qmv_get_device_error")
    return int(v.value)
