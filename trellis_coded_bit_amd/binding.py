"""Thin ctypes binding of libtrellis.so (argument marshalling only).

Every computation runs in the HIP library; this module checks dtypes, devices and
contiguity, allocates outputs and workspaces with torch, and passes raw device pointers
and the current HIP stream.  If the library is not built, loading fails loudly: there is
no fallback path.  Autograd records none of these calls: a result requires no gradient,
whatever its inputs do, and a program that trains calls the gradients' entry points itself.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import sys
import threading
from typing import Dict, List, Optional, Sequence, Tuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtrellis.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "trellis.h")

TRELLIS_OP_GEMV, TRELLIS_OP_GEMM, TRELLIS_OP_MOE_GEMV, TRELLIS_OP_GEMM_FP8 = 0, 1, 2, 3
TRELLIS_OP_MOE_MLP = 100  # workspace-cache key only (the C ABI has a dedicated size call)
STATUS = {0: "TRELLIS_OK", -1: "TRELLIS_EINVAL", -2: "TRELLIS_EALIGN", -3: "TRELLIS_EWORKSPACE",
          -4: "TRELLIS_EUNSUPPORTED", -5: "TRELLIS_EHIP"}


class TrellisError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class CLinear(ctypes.Structure):
    """Mirror of ``trellis_linear`` in include/trellis.h."""

    _fields_ = [
        ("code", ctypes.c_void_p),
        ("rin", ctypes.c_void_p),
        ("rout", ctypes.c_void_p),
        ("s_in", ctypes.c_void_p),
        ("s_out", ctypes.c_void_p),
        ("K", ctypes.c_int32),
        ("in_features", ctypes.c_int32),
        ("out_features", ctypes.c_int32),
        ("cb", ctypes.c_int32),
    ]


_lib = None
_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """Load libtrellis.so (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"{LIB_PATH} is not built; run `python -m trellis_coded_bit_amd.build`")
            L = ctypes.CDLL(LIB_PATH)
            vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            L.trellis_abi_version.restype = i32
            L.trellis_abi_version.argtypes = []
            L.trellis_last_error.restype = ctypes.c_char_p
            L.trellis_last_error.argtypes = []
            L.trellis_decode_tiles.restype = i32
            L.trellis_decode_tiles.argtypes = [vp, i32, i32, i32, vp, vp, vp]
            L.had128_scale.restype = i32
            L.had128_scale.argtypes = [vp, i32, i32, i32, vp, vp, i32, vp, i32, vp]
            L.trellis_workspace_bytes.restype = sz
            L.trellis_workspace_bytes.argtypes = [i32, ctypes.POINTER(CLinear), i32, i32]
            L.trellis_gemv.restype = i32
            L.trellis_gemv.argtypes = [ctypes.POINTER(CLinear), vp, i32, vp, vp, sz, vp]
            L.trellis_gemm.restype = i32
            L.trellis_gemm.argtypes = [ctypes.POINTER(CLinear), vp, i32, vp, vp, sz, vp]
            L.trellis_moe_gemv.restype = i32
            L.trellis_moe_gemv.argtypes = [vp, i32, vp, i32, i32, i32, vp, i32, vp, vp, i32, vp, vp, sz, vp]
            L.trellis_decode_tiles_e4m3.restype = i32
            L.trellis_decode_tiles_e4m3.argtypes = [vp, i32, i32, i32, vp, vp]
            L.trellis_gemm_fp8.restype = i32
            L.trellis_gemm_fp8.argtypes = [ctypes.POINTER(CLinear), vp, i32, vp, vp, sz, vp]
            L.trellis_encode_workspace_bytes.restype = sz
            L.trellis_encode_workspace_bytes.argtypes = [i32]
            L.trellis_encode_tiles.restype = i32
            L.trellis_encode_tiles.argtypes = [vp, i32, i32, i32, vp, vp, vp, sz, vp]
            L.trellis_moe_mlp_workspace_bytes.restype = sz
            L.trellis_moe_mlp_workspace_bytes.argtypes = [i32, i32, i32, i32]
            L.trellis_moe_mlp.restype = i32
            L.trellis_moe_mlp.argtypes = [vp, vp, i32, i32, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp,
                                          sz, vp]
            L.trellis_micro_cus.restype = i32
            L.trellis_micro_cus.argtypes = []
            L.trellis_micro_stream_read.restype = i32
            L.trellis_micro_stream_read.argtypes = [vp, sz, i32, vp, vp]
            L.trellis_micro_valu.restype = i32
            L.trellis_micro_valu.argtypes = [i32, i32, i32, vp, vp, vp, vp]
            L.trellis_micro_mfma.restype = i32
            L.trellis_micro_mfma.argtypes = [i32, i32, i32, vp, vp, vp, vp]
            L.trellis_gemv_list_workspace_bytes.restype = sz
            L.trellis_gemv_list_workspace_bytes.argtypes = [vp, i32, i32]
            L.trellis_gemv_list.restype = i32
            L.trellis_gemv_list.argtypes = [vp, i32, i32, vp, sz, vp]
            L.trellis_gemv_list_noalloc.restype = i32
            L.trellis_gemv_list_noalloc.argtypes = [vp, i32, i32, vp]
            i64, f32 = ctypes.c_int64, ctypes.c_float
            L.trellis_kv4_page_bytes.restype = sz
            L.trellis_kv4_page_bytes.argtypes = [i32, i32, i32]
            L.trellis_kv4_workspace_bytes.restype = sz
            L.trellis_kv4_workspace_bytes.argtypes = []
            L.trellis_kv4_attn_workspace_bytes.restype = sz
            L.trellis_kv4_attn_workspace_bytes.argtypes = [vp, vp, i32]
            L.trellis_kv4_pages_workspace_bytes.restype = sz
            L.trellis_kv4_pages_workspace_bytes.argtypes = [vp, i32]
            L.trellis_kv4_append.restype = i32
            L.trellis_kv4_append.argtypes = [vp, i32, vp, i32, vp, i64, i64, vp, i64, i64, vp, sz, vp]
            L.trellis_kv4_read.restype = i32
            L.trellis_kv4_read.argtypes = [vp, i32, vp, i32, vp, vp, vp, sz, vp]
            L.trellis_kv4_attn.restype = i32
            L.trellis_kv4_attn.argtypes = [vp, i32, vp, i32, vp, i64, i64, i32, f32, i32, i32, i32, vp, vp, vp, sz, vp]
            L.trellis_kv4_reserve.restype = i32
            L.trellis_kv4_reserve.argtypes = [vp, vp, vp, i32, i32, vp, vp, vp, i32, vp, sz, vp]
            L.trellis_kv4_fork.restype = i32
            L.trellis_kv4_fork.argtypes = [vp, vp, vp, i32, i32, vp, vp, vp, i32, vp, sz, vp]
            L.trellis_kv4_compact.restype = i32
            L.trellis_kv4_compact.argtypes = [vp, vp, vp, i32, i32, vp, vp, vp, i32, vp, vp, i32, vp, sz, vp]
            L.trellis_kv4_free.restype = i32
            L.trellis_kv4_free.argtypes = [vp, vp, vp, i32, i32, vp, vp, i32, vp, sz, vp]
            L.trellis_f8_norm.restype = i32
            L.trellis_f8_norm.argtypes = [i32, vp, i64, vp, vp, i32, i32, f32, vp, vp, vp, vp, vp]
            L.trellis_f8_silu_mul.restype = i32
            L.trellis_f8_silu_mul.argtypes = [i32, vp, i64, i32, i32, vp, vp, vp, vp]
            L.trellis_f8_gemm_workspace_bytes.restype = sz
            L.trellis_f8_gemm_workspace_bytes.argtypes = [vp, i32]
            L.trellis_f8_moe_gemm_workspace_bytes.restype = sz
            L.trellis_f8_moe_gemm_workspace_bytes.argtypes = [vp, i32]
            L.trellis_f8_gemm.restype = i32
            L.trellis_f8_gemm.argtypes = [vp, vp, i64, vp, i64, i32, i32, vp, i64, vp, sz, vp]
            L.trellis_f8_moe_gemm.restype = i32
            L.trellis_f8_moe_gemm.argtypes = [vp, vp, i64, vp, i64, i32, vp, vp, i32, i32, i32, vp, i64, vp, sz, vp]
            L.trellis_moe_sort_workspace_bytes.restype = sz
            L.trellis_moe_sort_workspace_bytes.argtypes = [i32, i32, i32]
            L.trellis_moe_rows_workspace_bytes.restype = sz
            L.trellis_moe_rows_workspace_bytes.argtypes = []
            L.trellis_moe_sort.restype = i32
            L.trellis_moe_sort.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, sz, vp]
            L.trellis_moe_gather.restype = i32
            L.trellis_moe_gather.argtypes = [vp, i64, i32, i64, vp, i32, i32, vp, vp, sz, vp]
            L.trellis_moe_combine.restype = i32
            L.trellis_moe_combine.argtypes = [i32, vp, i32, i32, vp, vp, i32, i32, vp, vp, vp, sz, vp]
            L.trellis_moe_combine_grad.restype = i32
            L.trellis_moe_combine_grad.argtypes = [i32, vp, vp, i32, i32, vp, vp, i32, i32, vp, vp, vp, sz, vp]
            L.trellis_validate_table.restype = i32
            L.trellis_validate_table.argtypes = [ctypes.POINTER(CLinear), i32, i32, i32, i32]
            _lib = L
    return _lib


def header_functions(header: str = HEADER) -> List[str]:
    """Names of the functions a header under include/ declares (default include/trellis.h)."""
    txt = open(header).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?(?:int|size_t|char\s*\*|const\s+char\s*\*)\s*\*?\s*(\w+)\s*\(", txt, flags=re.M)


def _check(status: int) -> None:
    if status != 0:
        raise TrellisError(status, lib().trellis_last_error().decode())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    """The current stream of the current device (without building a torch.cuda.Stream: that
    costs several microseconds a call)."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _req(t: torch.Tensor, dtype: torch.dtype, name: str, device=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ---------------------------------------------------------------------------------------
# Workspaces: zero-filled once, reused by back-to-back calls on one stream.
# ---------------------------------------------------------------------------------------

_ws: Dict[Tuple[int, int], torch.Tensor] = {}
# Buffers that a capture outgrew: nothing of them is recorded into the graph, and their error words
# count until they are cleared.
_ws_outgrown: Dict[Tuple[int, int], List[torch.Tensor]] = {}
# Buffers outgrown while a call of another thread (or the program) held them: what such a call is yet
# to set in an error word counts too.
_ws_held: Dict[Tuple[int, int], List[torch.Tensor]] = {}
_ws_lock = threading.RLock()  # (collected objects may call in while a buffer is made)


def _ws_replace(key: Tuple[int, int], w: torch.Tensor, old: List[torch.Tensor]) -> None:
    """w takes the place of old buffers; the error words of those that nobody else holds go on in it.
    (A call holds its workspace until it has reached the stream, and the fill that adds the word
    comes behind it there.)"""
    _ws[key] = w
    old += _ws_held.pop(key, [])
    held = []
    while old:
        o = old.pop()
        if sys.getrefcount(o) > 2:
            held.append(o)
        else:
            w[:4].bitwise_or_(o[:4])
        del o
    if held:
        _ws_held[key] = held


def workspace(nbytes: int, device: torch.device, op: int = 0) -> torch.Tensor:
    """One zero-filled workspace per (device, stream), grown on demand.  Every entry point
    leaves the reserved region at the start of a workspace as it found it, so all of them
    share one buffer (``op`` is accepted for compatibility and ignored), host threads on one
    stream too.  Its error word goes on with it when it grows.  (A graph should be given a
    workspace of the program's own: one made during a capture is cleared by every replay.)"""
    key = (device.index if device.index is not None else torch.cuda.current_device(), _stream())
    w = _ws.get(key)
    if w is None or w.numel() < nbytes:
        del w
        with _ws_lock:
            if key in _ws and _ws[key].numel() >= nbytes:  # (another thread's)
                return _ws[key]
            w = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
            if key in _ws and torch.cuda.is_current_stream_capturing():
                _ws_outgrown.setdefault(key, []).append(_ws[key])
                _ws[key] = w
            else:
                _ws_replace(key, w, [_ws.pop(key)] if key in _ws else [])
    return w


def _out(out: Optional[torch.Tensor], shape, device, dtype=torch.float16, name="out") -> torch.Tensor:
    """A new output tensor, or the caller's after checking dtype, device, contiguity and size
    (the kernels write exactly prod(shape) elements through its pointer)."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _req(out, dtype, name, device)
    n = 1
    for d in shape:
        n *= int(d)
    if out.numel() != n:
        raise ValueError(f"{name} has {out.numel()} elements, expected {n} (shape {tuple(shape)})")
    return out


def _ws_arg(ws: Optional[torch.Tensor], nb: int, device) -> torch.Tensor:
    if ws is None:
        return workspace(nb, device)
    _req(ws, torch.uint8, "ws", device)
    if ws.numel() < nb:
        raise ValueError(f"workspace of {ws.numel()} bytes < {nb}")
    return ws


class TrellisLinear:
    """Device tensors of one trellis-coded layer (y = x W, W [in, out])."""

    def __init__(self, code: torch.Tensor, rin: torch.Tensor, rout: torch.Tensor,
                 s_in: Optional[torch.Tensor], s_out: Optional[torch.Tensor], K: int, cb: int = 1):
        self.code, self.rin, self.rout, self.s_in, self.s_out, self.K = code, rin, rout, s_in, s_out, int(K)
        self.cb = int(cb)
        ti, tj, nw = code.shape
        self.in_features, self.out_features = 16 * ti, 16 * tj
        if nw != 16 * self.K:
            raise ValueError(f"code last dim {nw} != 16*K")
        dev = code.device
        _req(code, torch.int16, "code")
        _req(rin, torch.float16, "rin", dev)
        _req(rout, torch.float16, "rout", dev)
        if s_in is not None:
            _req(s_in, torch.float32, "s_in", dev)
        if s_out is not None:
            _req(s_out, torch.float32, "s_out", dev)
        self._c = None
        self._ws_bytes = {}

    @classmethod
    def from_host(cls, lin, device="cuda") -> "TrellisLinear":
        """From a ``synth.Linear`` (numpy arrays)."""
        t = lambda a: torch.from_numpy(a).to(device)
        return cls(t(lin.code), t(lin.rin), t(lin.rout), t(lin.s_in), t(lin.s_out), lin.K, getattr(lin, "cb", 1))

    def c(self) -> CLinear:
        if self._c is None:
            self._c = CLinear(_ptr(self.code), _ptr(self.rin), _ptr(self.rout), _ptr(self.s_in), _ptr(self.s_out),
                              self.K, self.in_features, self.out_features, self.cb)
        return self._c

    def workspace_bytes(self, op: int, batch_or_M: int) -> int:
        key = (op, batch_or_M)
        nb = self._ws_bytes.get(key)
        if nb is None:
            nb = lib().trellis_workspace_bytes(op, ctypes.byref(self.c()), batch_or_M, 0)
            self._ws_bytes[key] = nb
        return nb


# ---------------------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ---------------------------------------------------------------------------------------

def trellis_decode_tiles(code: torch.Tensor, K: int, want_states: bool = False):
    """code int16 [in/16, out/16, 16K] -> (w_hat fp16 [in, out], states uint16-as-int16 or None)."""
    _req(code, torch.int16, "code")
    ti, tj, nw = code.shape
    if nw != 16 * K:
        raise ValueError("code last dim must be 16*K")
    w = torch.empty((16 * ti, 16 * tj), dtype=torch.float16, device=code.device)
    st = torch.empty((ti, tj, 256), dtype=torch.int16, device=code.device) if want_states else None
    _check(lib().trellis_decode_tiles(code.data_ptr(), K, 16 * ti, 16 * tj, w.data_ptr(), _ptr(st), _stream()))
    return w, st


def had128_scale(x: torch.Tensor, r: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None,
                 post: bool = False, out_dtype: Optional[torch.dtype] = None,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = had(x*r*s) (post=False) or had(x)*r*s (post=True) over 128-blocks of the last axis."""
    if x.dtype not in (torch.float16, torch.float32):
        raise TypeError("x must be float16 or float32")
    _req(x, x.dtype, "x")
    n = x.shape[-1]
    rows = x.numel() // n if n else 0
    if r is not None:
        _req(r, torch.float16, "r", x.device)
    if s is not None:
        _req(s, torch.float32, "s", x.device)
    if out is not None and out.dtype not in (torch.float16, torch.float32):
        raise TypeError("out must be float16 or float32")
    out = _out(out, tuple(x.shape), x.device, out.dtype if out is not None else (out_dtype or x.dtype))
    _check(lib().had128_scale(x.data_ptr(), int(x.dtype == torch.float32), rows, n, _ptr(r), _ptr(s), int(post),
                              out.data_ptr(), int(out.dtype == torch.float32), _stream()))
    return out


def trellis_gemv(layer: TrellisLinear, x: torch.Tensor, out: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x fp16 [B, in] (B = 1..8) -> y fp16 [B, out].  ``ws``: optional uint8 workspace tensor
    (at least ``layer.workspace_bytes(TRELLIS_OP_GEMV, B)`` bytes), e.g. for graph capture."""
    _req(x, torch.float16, "x", layer.code.device)
    if x.numel() % layer.in_features:
        raise ValueError(f"x has {x.numel()} elements, not a multiple of in_features={layer.in_features}")
    x2 = x.reshape(-1, layer.in_features)
    B = x2.shape[0]
    out = _out(out, (B, layer.out_features), x.device)
    ws = _ws_arg(ws, layer.workspace_bytes(TRELLIS_OP_GEMV, B), x.device)
    _check(lib().trellis_gemv(ctypes.byref(layer.c()), x2.data_ptr(), B, out.data_ptr(), ws.data_ptr(), ws.numel(),
                              _stream()))
    return out


class CGemvItem(ctypes.Structure):
    """Mirror of ``trellis_gemv_item`` in include/trellis.h."""

    _fields_ = [("L", CLinear), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p)]


GEMV_LIST_MAX = 8


def _gemv_items(layers: Sequence[TrellisLinear], xs: Sequence[torch.Tensor], outs: Sequence[torch.Tensor]):
    items = (CGemvItem * len(layers))()
    for i, (l, x, y) in enumerate(zip(layers, xs, outs)):
        items[i].L = l.c()
        items[i].x = x.data_ptr()
        items[i].y = y.data_ptr()
    return items


def trellis_gemv_list_workspace_bytes(layers: Sequence[TrellisLinear], B: int) -> int:
    """Workspace bytes of trellis_gemv_list for these layers at batch B (fake x/y pointers:
    only shapes matter)."""
    items = (CGemvItem * len(layers))()
    for i, l in enumerate(layers):
        items[i].L = l.c()
        items[i].x = 0x1000 * (2 * i + 1) << 32
        items[i].y = 0x1000 * (2 * i + 2) << 32
    nb = lib().trellis_gemv_list_workspace_bytes(items, len(layers), B)
    if nb == 0:
        raise TrellisError(-4, lib().trellis_last_error().decode() or "unsupported list")
    return nb


def trellis_gemv_list(layers: Sequence[TrellisLinear], xs: Sequence[torch.Tensor],
                      outs: Optional[Sequence[Optional[torch.Tensor]]] = None,
                      ws: Optional[torch.Tensor] = None) -> List[torch.Tensor]:
    """One launch for several small-batch products: xs[p] fp16 [B, in_p] -> fp16 [B, out_p],
    the same B (1..8) for every layer."""
    n = len(layers)
    if n < 1 or n > GEMV_LIST_MAX or len(xs) != n:
        raise ValueError(f"1..{GEMV_LIST_MAX} layers with one input each expected")
    dev = layers[0].code.device
    x2s, B = [], None
    for l, x in zip(layers, xs):
        _req(x, torch.float16, "x", dev)
        if x.numel() % l.in_features:
            raise ValueError(f"x has {x.numel()} elements, not a multiple of in_features={l.in_features}")
        x2 = x.reshape(-1, l.in_features)
        if B is None:
            B = x2.shape[0]
        elif x2.shape[0] != B:
            raise ValueError("every input must have the same batch B")
        x2s.append(x2)
    outs = list(outs) if outs is not None else [None] * n
    if len(outs) != n:
        raise ValueError("one output (or None) per layer expected")
    ys = [_out(o, (B, l.out_features), dev) for o, l in zip(outs, layers)]
    items = _gemv_items(layers, x2s, ys)
    nb = lib().trellis_gemv_list_workspace_bytes(items, n, B)
    if nb == 0:
        _check(lib().trellis_gemv_list(items, n, B, None, 0, _stream()))
    ws = _ws_arg(ws, nb, dev)
    _check(lib().trellis_gemv_list(items, n, B, ws.data_ptr(), ws.numel(), _stream()))
    return ys


def trellis_gemm(layer: TrellisLinear, x: torch.Tensor, out: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x fp16 [M, in] -> y fp16 [M, out]."""
    _req(x, torch.float16, "x", layer.code.device)
    if x.dim() != 2 or x.shape[1] != layer.in_features:
        raise ValueError(f"x must be [M, {layer.in_features}]")
    M = x.shape[0]
    out = _out(out, (M, layer.out_features), x.device)
    ws = _ws_arg(ws, layer.workspace_bytes(TRELLIS_OP_GEMM, M), x.device)
    _check(lib().trellis_gemm(ctypes.byref(layer.c()), x.data_ptr(), M, out.data_ptr(), ws.data_ptr(), ws.numel(),
                              _stream()))
    return out


def trellis_decode_tiles_e4m3(code: torch.Tensor, K: int) -> torch.Tensor:
    """code int16 [in/16, out/16, 16K] -> E4M3 codes uint8 [in, out] (the cb = 2 weights)."""
    _req(code, torch.int16, "code")
    ti, tj, nw = code.shape
    if nw != 16 * K:
        raise ValueError("code last dim must be 16*K")
    w8 = torch.empty((16 * ti, 16 * tj), dtype=torch.uint8, device=code.device)
    _check(lib().trellis_decode_tiles_e4m3(code.data_ptr(), K, 16 * ti, 16 * tj, w8.data_ptr(), _stream()))
    return w8


def trellis_gemm_fp8(layer: TrellisLinear, x: torch.Tensor, out: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x fp16 [M, in] -> y fp16 [M, out] on the FP8 matrix cores (layer.cb must be 2)."""
    _req(x, torch.float16, "x", layer.code.device)
    if x.dim() != 2 or x.shape[1] != layer.in_features:
        raise ValueError(f"x must be [M, {layer.in_features}]")
    M = x.shape[0]
    out = _out(out, (M, layer.out_features), x.device)
    ws = _ws_arg(ws, layer.workspace_bytes(TRELLIS_OP_GEMM_FP8, M), x.device)
    _check(lib().trellis_gemm_fp8(ctypes.byref(layer.c()), x.data_ptr(), M, out.data_ptr(), ws.data_ptr(),
                                  ws.numel(), _stream()))
    return out


def trellis_encode_tiles(targets: torch.Tensor, K: int, cb: int = 1, want_states: bool = False,
                         ws: Optional[torch.Tensor] = None):
    """targets f32 [T, 16, 16] -> (code int16 [T, 16K], states uint16-as-int16 [T, 256] or None)."""
    _req(targets, torch.float32, "targets")
    if targets.dim() != 3 or tuple(targets.shape[1:]) != (16, 16):
        raise ValueError("targets must be [T, 16, 16]")
    T = targets.shape[0]
    code = torch.empty((T, 16 * K), dtype=torch.int16, device=targets.device)
    st = torch.empty((T, 256), dtype=torch.int16, device=targets.device) if want_states else None
    nb = lib().trellis_encode_workspace_bytes(T)
    if ws is None:
        ws = torch.empty(max(nb, 256), dtype=torch.uint8, device=targets.device)
    elif ws.numel() < nb:
        raise ValueError(f"workspace of {ws.numel()} bytes < {nb}")
    _check(lib().trellis_encode_tiles(targets.data_ptr(), T, K, cb, code.data_ptr(), _ptr(st), ws.data_ptr(),
                                      ws.numel(), _stream()))
    return code, st


class ExpertTable:
    """A device-resident table of trellis_linear descriptors (uniform in/out, per-entry K)."""

    def __init__(self, layers: Sequence[TrellisLinear], shared_side: int = -1, device="cuda"):
        self.layers = list(layers)  # keeps the tensors alive
        self.in_features = self.layers[0].in_features
        self.out_features = self.layers[0].out_features
        host = (CLinear * len(self.layers))(*[l.c() for l in self.layers])
        for i, l in enumerate(self.layers):
            if shared_side == 0:
                host[i].rin, host[i].s_in = None, None
            if shared_side == 1:
                host[i].rout, host[i].s_out = None, None
        _check(lib().trellis_validate_table(host, len(self.layers), self.in_features, self.out_features, shared_side))
        raw = bytes(host)
        self.table = torch.frombuffer(bytearray(raw), dtype=torch.uint8).to(device)
        self.E = len(self.layers)
        self._ws_bytes = {}

    def workspace_bytes(self, n: int) -> int:
        nb = self._ws_bytes.get(n)
        if nb is None:
            probe = CLinear(None, None, None, None, None, 2, self.in_features, self.out_features, 1)
            nb = lib().trellis_workspace_bytes(TRELLIS_OP_MOE_GEMV, ctypes.byref(probe), 1, n)
            self._ws_bytes[n] = nb
        return nb


def trellis_moe_gemv(table: ExpertTable, routed: torch.Tensor, x: torch.Tensor, x_per_expert: bool,
                     shared_r: Optional[torch.Tensor] = None, shared_s: Optional[torch.Tensor] = None,
                     shared_side: int = -1, out: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """routed int32 [n] (device); x fp16 [in] or [n, in]; returns y fp16 [n, out]."""
    _req(routed, torch.int32, "routed")
    dev = routed.device
    _req(x, torch.float16, "x", dev)
    n = routed.numel()
    if x.numel() != (n if x_per_expert else 1) * table.in_features:
        raise ValueError(f"x must have {'n*' if x_per_expert else ''}in = "
                         f"{(n if x_per_expert else 1) * table.in_features} elements")
    for name, v, dt in (("shared_r", shared_r, torch.float16), ("shared_s", shared_s, torch.float32)):
        if v is not None:
            _req(v, dt, name, dev)
            side_n = table.in_features if shared_side == 0 else table.out_features
            if v.numel() != side_n:
                raise ValueError(f"{name} must have {side_n} elements")
    out = _out(out, (n, table.out_features), dev)
    ws = _ws_arg(ws, table.workspace_bytes(n), dev)
    _check(lib().trellis_moe_gemv(table.table.data_ptr(), table.E, routed.data_ptr(), n, table.in_features,
                                  table.out_features, x.data_ptr(), int(x_per_expert), _ptr(shared_r),
                                  _ptr(shared_s), shared_side, out.data_ptr(), ws.data_ptr(), ws.numel(), _stream()))
    return out


def _error_words(ws: Optional[torch.Tensor], device) -> List[torch.Tensor]:
    if ws is not None:
        return [ws]
    key = (torch.device(device).index or 0, _stream())
    with _ws_lock:
        return ([_ws[key]] if key in _ws else []) + _ws_outgrown.get(key, []) + _ws_held.get(key, [])


def error_word(ws: Optional[torch.Tensor] = None, device="cuda") -> int:
    """The error word of a workspace (default: the current stream's shared one); it is
    sticky (bit 1: a bad routed id or table entry was skipped; bit 2: a bounded wait ran
    out; bits 4 and 8: the key/value cache's, a bad place and too few free pages).
    Synchronises."""
    word = 0
    for w in _error_words(ws, device):
        word |= int(w[:4].view(torch.int32).item())
    return word


def clear_error_word(ws: Optional[torch.Tensor] = None, device="cuda") -> None:
    """Clear a workspace's error word (a fill on the current stream; graph-safe)."""
    for w in _error_words(ws, device):
        w[:4].zero_()


class MoEMLPTables:
    """Device tables of a routed-expert MLP layer: gate/up slices [E][2H] (entry e*2H + h is
    slice h of gate_e, e*2H + H + h slice h of up_e) and down [E]."""

    def __init__(self, gate: Sequence[Sequence[TrellisLinear]], up: Sequence[Sequence[TrellisLinear]],
                 down: Sequence[TrellisLinear], device="cuda"):
        self.E = len(down)
        self.halves = len(gate[0])
        entries = []
        for e in range(self.E):
            if len(gate[e]) != self.halves or len(up[e]) != self.halves:
                raise ValueError(f"expert {e}: every expert needs {self.halves} gate and up slices")
            entries += list(gate[e]) + list(up[e])
        self.gate_up = ExpertTable(entries, shared_side=0, device=device)
        self.down = ExpertTable(down, shared_side=1, device=device)
        self.hidden = self.gate_up.in_features
        self.inter = self.gate_up.out_features * self.halves
        if self.down.in_features != self.inter or self.down.out_features != self.hidden:
            raise ValueError("down must map inter -> hidden")

    @classmethod
    def from_host(cls, layer, device="cuda") -> "MoEMLPTables":
        """From a ``synth.MoEMLPLayer``; the shared hidden-side arrays are uploaded once and
        every descriptor points at that one copy."""
        t = lambda a: torch.from_numpy(a).to(device)
        r_hi, s_hi = t(layer.r_hidden_in), t(layer.s_hidden_in)
        r_ho, s_ho = t(layer.r_hidden_out), t(layer.s_hidden_out)
        dev = lambda l, rin, s_in, rout, s_out: TrellisLinear(t(l.code), rin, rout, s_in, s_out, l.K,
                                                              getattr(l, "cb", 1))
        E = len(layer.down)
        gate = [[dev(l, r_hi, s_hi, t(l.rout), t(l.s_out)) for l in layer.gate[e]] for e in range(E)]
        up = [[dev(l, r_hi, s_hi, t(l.rout), t(l.s_out)) for l in layer.up[e]] for e in range(E)]
        down = [dev(layer.down[e], t(layer.down[e].rin), t(layer.down[e].s_in), r_ho, s_ho) for e in range(E)]
        obj = cls(gate, up, down, device=device)
        obj.r_hidden_in, obj.s_hidden_in, obj.r_hidden_out, obj.s_hidden_out = r_hi, s_hi, r_ho, s_ho
        return obj

    def workspace_bytes(self, n: int) -> int:
        nb = lib().trellis_moe_mlp_workspace_bytes(self.hidden, self.inter, self.halves, n)
        if nb == 0:
            raise ValueError(f"invalid MLP sizes for n={n}")
        return nb


def trellis_moe_mlp(tables: MoEMLPTables, routed: torch.Tensor, router_w: torch.Tensor, x: torch.Tensor,
                    r_hidden_in: torch.Tensor, s_hidden_in: Optional[torch.Tensor],
                    r_hidden_out: torch.Tensor, s_hidden_out: Optional[torch.Tensor],
                    out: Optional[torch.Tensor] = None, act: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """routed int32 [n], router_w f32 [n], x fp16 [hidden] -> y fp16 [hidden].
    ``act``: optional fp16 [n, inter] receiving silu(gate x) * up x."""
    _req(routed, torch.int32, "routed")
    dev = routed.device
    _req(router_w, torch.float32, "router_w", dev)
    _req(x, torch.float16, "x", dev)
    n = routed.numel()
    if router_w.numel() != n:
        raise ValueError("router_w must have one weight per routed expert")
    if x.numel() != tables.hidden:
        raise ValueError(f"x must have {tables.hidden} elements")
    for name, v, dt in (("r_hidden_in", r_hidden_in, torch.float16), ("r_hidden_out", r_hidden_out, torch.float16),
                        ("s_hidden_in", s_hidden_in, torch.float32), ("s_hidden_out", s_hidden_out, torch.float32)):
        if v is not None:
            _req(v, dt, name, dev)
            if v.numel() != tables.hidden:
                raise ValueError(f"{name} must have {tables.hidden} elements")
    out = _out(out, (tables.hidden,), dev)
    if act is not None:
        _req(act, torch.float16, "act", dev)
        if act.numel() != n * tables.inter:
            raise ValueError(f"act must have n*inter = {n * tables.inter} elements")
    ws = _ws_arg(ws, tables.workspace_bytes(n), dev)
    _check(lib().trellis_moe_mlp(tables.gate_up.table.data_ptr(), tables.down.table.data_ptr(), tables.E,
                                 tables.halves, routed.data_ptr(), router_w.data_ptr(), n, tables.hidden,
                                 tables.inter, x.data_ptr(), _ptr(r_hidden_in), _ptr(s_hidden_in),
                                 _ptr(r_hidden_out), _ptr(s_hidden_out), _ptr(act), out.data_ptr(),
                                 ws.data_ptr(), ws.numel(), _stream()))
    return out


# ---------------------------------------------------------------------------------------
# The paged 4-bit key/value cache (include/trellis_kv4.h)
# ---------------------------------------------------------------------------------------

class CKV4Cache(ctypes.Structure):
    """Mirror of ``trellis_kv4_cache`` in include/trellis_kv4.h."""

    _fields_ = [("pool", ctypes.c_void_p), ("n_layers", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class CKV4Batch(ctypes.Structure):
    """Mirror of ``trellis_kv4_batch`` in include/trellis_kv4.h."""

    _fields_ = [("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("cu", ctypes.c_void_p), ("n_slots", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("n_seq", ctypes.c_int32), ("rows", ctypes.c_int32)]


_KV4_DTYPE = {torch.float16: 0, torch.bfloat16: 1}


@functools.lru_cache(maxsize=None)
def trellis_kv4_page_bytes(page_size: int, n_kv_heads: int, head_dim: int) -> int:
    """Bytes of one page of one layer."""
    nb = lib().trellis_kv4_page_bytes(page_size, n_kv_heads, head_dim)
    if nb == 0:
        raise ValueError(f"page_size={page_size} n_kv_heads={n_kv_heads} head_dim={head_dim}: pages of 16, 32, 64, 128 "
                         "or 256 tokens, 1..1024 heads of 128 or 256 expected")
    return nb


@functools.lru_cache(maxsize=None)
def _kv4_ws_bytes() -> int:
    return lib().trellis_kv4_workspace_bytes()


class KV4Cache:
    """A cache of keys and values in 4 bits: ``pool`` uint8 [n_layers, n_pages, page_bytes] on a
    GPU.  The page table (int32 [slots, max_pages]), the lengths (int32 [slots]) and the pages'
    reference counts (int32 [n_pages]) are the caller's tensors, passed to each call."""

    def __init__(self, pool: torch.Tensor, page_size: int, n_kv_heads: int, head_dim: int):
        nb = trellis_kv4_page_bytes(page_size, n_kv_heads, head_dim)
        _req(pool, torch.uint8, "pool")
        if pool.dim() != 3 or pool.shape[2] != nb or pool.shape[0] < 1 or pool.shape[1] < 1:
            raise ValueError(f"pool must be [n_layers, n_pages, {nb}], got {tuple(pool.shape)}")
        self.pool, self.page_size, self.n_kv_heads, self.head_dim = pool, page_size, n_kv_heads, head_dim
        self.n_layers, self.n_pages = pool.shape[0], pool.shape[1]
        self.device = pool.device
        self._c = CKV4Cache(pool.data_ptr(), self.n_layers, self.n_pages, page_size, n_kv_heads, head_dim)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def allocate(cls, n_layers: int, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int,
                 device="cuda") -> "KV4Cache":
        nb = trellis_kv4_page_bytes(page_size, n_kv_heads, head_dim)
        return cls(torch.zeros((n_layers, n_pages, nb), dtype=torch.uint8, device=device), page_size, n_kv_heads, head_dim)


def _kv4_int(t: torch.Tensor, name: str, device) -> None:
    """_req for the int32 tensors of a call, the usual case first."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.device == device and t.is_contiguous()):
        _req(t, torch.int32, name, device)


def _kv4_ws(ws: Optional[torch.Tensor], nb: int, device, stream: int) -> torch.Tensor:
    """_ws_arg with the stream at hand."""
    if ws is None:
        w = _ws.get((device.index, stream))
        return w if w is not None and w.numel() >= nb else workspace(nb, device)
    return _ws_arg(ws, nb, device)


def _kv4_state(cache: KV4Cache, table: torch.Tensor, lens: torch.Tensor) -> None:
    _kv4_int(table, "table", cache.device)
    _kv4_int(lens, "lens", cache.device)
    if table.dim() != 2 or lens.numel() != table.shape[0]:
        raise ValueError(f"table must be [slots, max_pages] with one length per slot, got {tuple(table.shape)} and "
                         f"{lens.numel()} lengths")


def _kv4_batch(cache: KV4Cache, table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor,
               slots: Optional[torch.Tensor], rows: int) -> CKV4Batch:
    _kv4_state(cache, table, lens)
    _kv4_int(cu, "cu", cache.device)
    n_seq = cu.numel() - 1
    if slots is not None:
        _kv4_int(slots, "slots", cache.device)
        if slots.numel() != n_seq:
            raise ValueError(f"slots must have one entry per sequence ({n_seq}), got {slots.numel()}")
    elif n_seq > lens.numel():
        raise ValueError(f"{n_seq} sequences over {lens.numel()} slots")
    if n_seq < 0:
        raise ValueError("cu must have one entry more than there are sequences")
    return CKV4Batch(table.data_ptr(), lens.data_ptr(), _ptr(slots), cu.data_ptr(), table.shape[0], table.shape[1], n_seq,
                     rows)


def _kv4_rows(cache: KV4Cache, x: torch.Tensor, heads: Optional[int], name: str):
    """Checks a [rows, heads, head_dim] tensor whose vectors are contiguous; its strides."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype not in _KV4_DTYPE:
        raise TypeError(f"{name} must be float16 or bfloat16, got {x.dtype}")
    if x.device != cache.device:
        raise ValueError(f"{name} is on {x.device}, expected {cache.device}")
    if x.dim() != 3 or x.shape[2] != cache.head_dim or (heads is not None and x.shape[1] != heads):
        raise ValueError(f"{name} must be [rows, {heads if heads is not None else 'heads'}, {cache.head_dim}], got "
                         f"{tuple(x.shape)}")
    row, head, last = x.stride()
    if last != 1:
        raise ValueError(f"{name}: each head's vector must be contiguous")
    # (one row or head: its stride is used for nothing and may be any number)
    return row if x.shape[0] > 1 else 0, head if x.shape[1] > 1 else 0


def trellis_kv4_append(cache: KV4Cache, layer: int, table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor,
                       k: torch.Tensor, v: torch.Tensor, slots: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None) -> None:
    """Quantise new keys and values, [rows, n_kv_heads, head_dim] fp16 or bf16 (slices of a
    fused projection's output are fine), into one layer.  Sequence b (slot ``slots[b]``, or b)
    has the rows cu[b] .. cu[b+1]-1, its last tokens; ``lens`` already counts them."""
    k_row, k_head = _kv4_rows(cache, k, cache.n_kv_heads, "k")
    v_row, v_head = _kv4_rows(cache, v, cache.n_kv_heads, "v")
    if v.dtype != k.dtype or v.shape[0] != k.shape[0]:
        raise ValueError("k and v must have the same type and number of rows")
    b = _kv4_batch(cache, table, lens, cu, slots, k.shape[0])
    stream = _stream()
    ws = _kv4_ws(ws, _kv4_ws_bytes(), cache.device, stream)
    _check(lib().trellis_kv4_append(cache._ref, layer, ctypes.byref(b), _KV4_DTYPE[k.dtype], k.data_ptr(), k_row, k_head,
                                    v.data_ptr(), v_row, v_head, ws.data_ptr(), ws.numel(), stream))


def trellis_kv4_read(cache: KV4Cache, layer: int, table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor, rows: int,
                     dtype: torch.dtype = torch.float16, slots: Optional[torch.Tensor] = None,
                     out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, ws: Optional[torch.Tensor] = None):
    """The keys and values that the cache holds for each sequence's last cu[b+1] - cu[b]
    tokens, rotated back: (k, v), each [rows, n_kv_heads, head_dim]."""
    if dtype not in _KV4_DTYPE:
        raise TypeError(f"dtype must be float16 or bfloat16, got {dtype}")
    shape = (rows, cache.n_kv_heads, cache.head_dim)
    k, v = (_out(o, shape, cache.device, dtype, n) for o, n in zip(out if out is not None else (None, None), ("k", "v")))
    b = _kv4_batch(cache, table, lens, cu, slots, rows)
    stream = _stream()
    ws = _kv4_ws(ws, _kv4_ws_bytes(), cache.device, stream)
    _check(lib().trellis_kv4_read(cache._ref, layer, ctypes.byref(b), _KV4_DTYPE[dtype], k.data_ptr(), v.data_ptr(),
                                  ws.data_ptr(), ws.numel(), stream))
    return k, v


def trellis_kv4_attn_workspace_bytes(cache: KV4Cache, table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor,
                                     rows: int, n_q_heads: int, slots: Optional[torch.Tensor] = None) -> int:
    """Workspace bytes of trellis_kv4_attn for these sizes."""
    return _kv4_attn_bytes(cache, _kv4_batch(cache, table, lens, cu, slots, rows), n_q_heads)


# Workspace sizes of attention by the sizes they follow from (not by tensors).
_kv4_attn_nb: Dict[Tuple[int, ...], int] = {}


def _kv4_attn_bytes(cache: KV4Cache, b: CKV4Batch, n_q_heads: int) -> int:
    key = (cache.page_size, cache.n_kv_heads, cache.head_dim, b.max_pages, b.n_seq, b.rows, n_q_heads, cache.device.index)
    nb = _kv4_attn_nb.get(key)
    if nb is None:
        nb = lib().trellis_kv4_attn_workspace_bytes(cache._ref, ctypes.byref(b), n_q_heads)
        if nb == 0:
            raise TrellisError(-1, lib().trellis_last_error().decode())
        if len(_kv4_attn_nb) >= 4096:  # (a long-running server sees many row counts)
            _kv4_attn_nb.clear()
        _kv4_attn_nb[key] = nb
    return nb


def trellis_kv4_attn(cache: KV4Cache, layer: int, table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor,
                     q: torch.Tensor, window: int = 0, sinks: int = 0, scale: Optional[float] = None, max_q: int = 0,
                     slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention of q [rows, n_q_heads, head_dim] (fp16 or bf16) over the cache: row
    cu[b] + i is sequence b's token at lens - (cu[b+1] - cu[b]) + i and sees the keys up to
    itself, with ``window`` only the last ``window`` of them and the first ``sinks`` tokens.
    ``scale`` defaults to head_dim ** -0.5.  ``max_q``: a bound on a sequence's rows if the
    caller knows one (it chooses kernels).  ``lse``: optional f32 [rows, n_q_heads] output, the
    logarithm of each softmax's denominator."""
    q_row, q_head = _kv4_rows(cache, q, None, "q")
    rows, heads = q.shape[0], q.shape[1]
    out = _out(out, (rows, heads, cache.head_dim), cache.device, q.dtype)
    if lse is not None:
        _out(lse, (rows, heads), cache.device, torch.float32, "lse")
    b = _kv4_batch(cache, table, lens, cu, slots, rows)
    stream = _stream()
    ws = _kv4_ws(ws, _kv4_attn_bytes(cache, b, heads), cache.device, stream)
    _check(lib().trellis_kv4_attn(cache._ref, layer, ctypes.byref(b), _KV4_DTYPE[q.dtype], q.data_ptr(), q_row, q_head,
                                  heads, cache.head_dim ** -0.5 if scale is None else scale, window, sinks, max_q,
                                  out.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(), stream))
    return out


def _kv4_pages(cache: KV4Cache, table: torch.Tensor, lens: torch.Tensor, ref: torch.Tensor, **lists) -> int:
    """Checks the page operations' tensors; the number of items (the first list's length)."""
    _kv4_state(cache, table, lens)
    _kv4_int(ref, "ref", cache.device)
    if ref.numel() != cache.n_pages:
        raise ValueError(f"ref must have one count per page ({cache.n_pages}), got {ref.numel()}")
    n = None
    for name, (t, extra) in lists.items():
        if t is None:
            continue
        _kv4_int(t, name, cache.device)
        if n is None:
            n = t.numel()
        elif t.numel() != n + extra:
            raise ValueError(f"{name} must have {n + extra} entries, got {t.numel()}")
    return n


def trellis_kv4_reserve(cache: KV4Cache, table: torch.Tensor, lens: torch.Tensor, ref: torch.Tensor, add: torch.Tensor,
                        slots: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> None:
    """lens[slots[i]] += add[i] (slots None: slot i) with the pages that takes, lowest first.
    If there are not enough, nothing changes and bit 8 of the error word is set."""
    n = _kv4_pages(cache, table, lens, ref, add=(add, 0), slots=(slots, 0))
    stream = _stream()
    ws = _kv4_ws(ws, lib().trellis_kv4_pages_workspace_bytes(cache._ref, n), cache.device, stream)
    _check(lib().trellis_kv4_reserve(cache._ref, table.data_ptr(), lens.data_ptr(), table.shape[0], table.shape[1],
                                     ref.data_ptr(), _ptr(slots), add.data_ptr(), n, ws.data_ptr(), ws.numel(), stream))


def trellis_kv4_fork(cache: KV4Cache, table: torch.Tensor, lens: torch.Tensor, ref: torch.Tensor, src: torch.Tensor,
                     dst: torch.Tensor, ws: Optional[torch.Tensor] = None) -> None:
    """Slot dst[i] becomes a copy of slot src[i]: full pages shared, a partly filled last page
    copied.  What dst held is released."""
    n = _kv4_pages(cache, table, lens, ref, src=(src, 0), dst=(dst, 0))
    stream = _stream()
    ws = _kv4_ws(ws, lib().trellis_kv4_pages_workspace_bytes(cache._ref, n), cache.device, stream)
    _check(lib().trellis_kv4_fork(cache._ref, table.data_ptr(), lens.data_ptr(), table.shape[0], table.shape[1],
                                  ref.data_ptr(), src.data_ptr(), dst.data_ptr(), n, ws.data_ptr(), ws.numel(), stream))


def trellis_kv4_compact(cache: KV4Cache, table: torch.Tensor, lens: torch.Tensor, ref: torch.Tensor, src: torch.Tensor,
                        dst: torch.Tensor, keep: torch.Tensor, keep_cu: torch.Tensor,
                        ws: Optional[torch.Tensor] = None) -> None:
    """Slot dst[i] becomes the tokens keep[keep_cu[i]:keep_cu[i+1]] of slot src[i] (positions),
    packed into new pages; dst[i] may be src[i].  What dst held is released."""
    n = _kv4_pages(cache, table, lens, ref, src=(src, 0), dst=(dst, 0), keep_cu=(keep_cu, 1))
    _req(keep, torch.int32, "keep", cache.device)
    stream = _stream()
    ws = _kv4_ws(ws, lib().trellis_kv4_pages_workspace_bytes(cache._ref, n), cache.device, stream)
    _check(lib().trellis_kv4_compact(cache._ref, table.data_ptr(), lens.data_ptr(), table.shape[0], table.shape[1],
                                     ref.data_ptr(), src.data_ptr(), dst.data_ptr(), n, keep.data_ptr(),
                                     keep_cu.data_ptr(), keep.numel(), ws.data_ptr(), ws.numel(), stream))


def trellis_kv4_free(cache: KV4Cache, table: torch.Tensor, lens: torch.Tensor, ref: torch.Tensor, slots: torch.Tensor,
                     ws: Optional[torch.Tensor] = None) -> None:
    """Release slots: their pages' counts drop, their lengths become 0."""
    n = _kv4_pages(cache, table, lens, ref, slots=(slots, 0))
    stream = _stream()
    ws = _kv4_ws(ws, _kv4_ws_bytes(), cache.device, stream)
    _check(lib().trellis_kv4_free(cache._ref, table.data_ptr(), lens.data_ptr(), table.shape[0], table.shape[1],
                                  ref.data_ptr(), slots.data_ptr(), n, ws.data_ptr(), ws.numel(), stream))


# ---------------------------------------------------------------------------------------
# Block-scaled FP8 (include/trellis_f8.h) and routed tokens (include/trellis_route.h)
# ---------------------------------------------------------------------------------------

class CF8Linear(ctypes.Structure):
    """Mirror of ``trellis_f8_linear`` in include/trellis_f8.h."""

    _fields_ = [("w", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("n_experts", ctypes.c_int32),
                ("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32)]


_E4M3 = torch.float8_e4m3fn
_F8_DTYPE = {torch.float16: 0, torch.bfloat16: 1}


def _f8_blocks(n: int) -> int:
    return (n + 127) // 128


def _i31(n: int, name: str) -> int:
    """A size that the C call takes in 32 bits (ctypes would cut it off)."""
    if n >> 31:
        raise ValueError(f"{name}={n} not in 0..2^31-1")
    return n


def _f8_rows(t: torch.Tensor, name: str, dtype: Optional[torch.dtype] = None, device=None,
             cols: Optional[int] = None) -> int:
    """Checks a [rows, cols] tensor on the current device whose rows are contiguous (16-bit if
    no dtype is given); its row stride."""
    # the usual case first: what is checked costs as much time as a short call's kernel
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 2 and t.get_device() == torch._C._cuda_getDevice():
        d = t.dtype
        if d is dtype or (dtype is None and d in _F8_DTYPE):
            rows, n = t.shape
            row, last = t.stride()
            if ((last == 1 or n <= 1) and (cols is None or n == cols) and (device is None or t.device == device)
                    and not (rows | n) >> 31):
                return row if rows > 1 else n
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype and (dtype is not None or t.dtype not in _F8_DTYPE):
        raise TypeError(f"{name} must be {'float16 or bfloat16' if dtype is None else dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if t.get_device() != torch._C._cuda_getDevice() or (device is not None and t.device != device):
        raise ValueError(f"{name} is on {t.device}: the current device is cuda:{torch._C._cuda_getDevice()}")
    if t.dim() != 2 or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} must be [rows, {'n' if cols is None else cols}], got {tuple(t.shape)}")
    _i31(t.shape[0], f"rows of {name}")
    _i31(t.shape[1], f"columns of {name}")
    raise ValueError(f"{name}: each row must be contiguous")


def _f8_ws(ws: Optional[torch.Tensor], nb: int, device) -> torch.Tensor:
    return _kv4_ws(ws, nb, device, _stream())


# A new tensor on the current device, for half of what torch.empty's argument parsing takes.  It passes
# by what a program may put between: modes that see every call, and the fill of new memory that
# deterministic algorithms ask for.  Where one of these is on, torch.empty is called.
def _find_empty_cuda():
    try:
        C = torch._C
        return C._dynamo.guards._empty_strided_cuda, C._len_torch_dispatch_stack, C._len_torch_function_stack, C._get_deterministic_algorithms
    except AttributeError:
        return None, None, None, None


_empty_cuda, _dispatch_modes, _function_modes, _deterministic = _find_empty_cuda()


def _new(shape: Tuple[int, ...], stride: Tuple[int, ...], dtype: torch.dtype, device) -> torch.Tensor:
    if _empty_cuda is None or _dispatch_modes() or _function_modes() or _deterministic():
        return torch.empty(shape, dtype=dtype, device=device)
    return _empty_cuda(shape, stride, dtype)


def _new1(n: int, dtype: torch.dtype, device) -> torch.Tensor:
    return _new((n,), (1,), dtype, device)


def _new2(rows: int, n: int, dtype: torch.dtype, device) -> torch.Tensor:
    return _new((rows, n), (n, 1), dtype, device)


def _out1(t: Optional[torch.Tensor], n: int, device, dtype: torch.dtype, name: str) -> torch.Tensor:
    return _new1(n, dtype, device) if t is None else _out(t, (n,), device, dtype, name)


def _out2(t: Optional[torch.Tensor], rows: int, n: int, device, dtype: torch.dtype, name: str = "out") -> torch.Tensor:
    """_out for [rows, n] on the current device."""
    return _new2(rows, n, dtype, device) if t is None else _out(t, (rows, n), device, dtype, name)


def _f8_out(q, scale, rows: int, n: int, device):
    return (_out2(q, rows, n, device, _E4M3, "q"), _out2(scale, rows, (n + 127) // 128, device, torch.float32, "scale"))


def trellis_f8_norm(x: torch.Tensor, gamma: Optional[torch.Tensor], eps: float, residual: Optional[torch.Tensor] = None,
                    quantize: bool = True, h: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                    scale: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """Root-mean-square norm of h = x + residual, x [rows, n] fp16 or bf16 (a slice with its own
    row stride is fine), residual [rows, n], gamma [n] of the same type or None: (q, scale, h),
    the E4M3 codes (float8_e4m3fn [rows, n]) with one f32 scale per 128 channels, and h rounded
    (the next residual; ``h=residual`` updates it in place), None if there is no residual and no
    ``h``.  ``y``: optional 16-bit output of the norm itself; with ``quantize=False`` it is the
    only one (q and scale are None, y is made if not given) and takes their place: (y, h)."""
    x_row = _f8_rows(x, "x")
    rows, n = x.shape
    dev, dtype = x.device, x.dtype
    r = g = None
    if residual is not None:
        _req(residual, dtype, "residual", dev)
        if residual.shape != x.shape:
            raise ValueError(f"residual must be {(rows, n)}, got {tuple(residual.shape)}")
        r = residual.data_ptr()
    if gamma is not None:
        _req(gamma, dtype, "gamma", dev)
        if gamma.numel() != n:
            raise ValueError(f"gamma must have {n} elements")
        g = gamma.data_ptr()
    if residual is not None or h is not None:
        h = _out2(h, rows, n, dev, dtype, "h")
    if quantize:
        q, scale = _f8_out(q, scale, rows, n, dev)
    elif q is not None or scale is not None:
        raise ValueError("q and scale are not written with quantize=False")
    if y is not None or not quantize:
        y = _out2(y, rows, n, dev, dtype, "y")
    st = lib().trellis_f8_norm(_F8_DTYPE[dtype], x.data_ptr(), x_row, r, g, rows, n, eps, None if h is None else h.data_ptr(),
                               _ptr(q), _ptr(scale), None if y is None else y.data_ptr(), _stream())
    if st:
        _check(st)
    return (q, scale, h) if quantize else (y, h)


def trellis_f8_silu_mul(x: torch.Tensor, quantize: bool = True, q: Optional[torch.Tensor] = None,
                        scale: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """silu(g) * u of x [rows, 2n] fp16 or bf16 with g in its first n columns: (q, scale), E4M3
    codes with one f32 scale per 128 channels.  ``y``: optional 16-bit output; with
    ``quantize=False`` the only one, returned."""
    x_row = _f8_rows(x, "x")
    rows, n = x.shape
    if n % 2:
        raise ValueError(f"x must have an even number of columns, got {n}")
    n //= 2
    if quantize:
        q, scale = _f8_out(q, scale, rows, n, x.device)
    elif q is not None or scale is not None:
        raise ValueError("q and scale are not written with quantize=False")
    if y is not None or not quantize:
        y = _out2(y, rows, n, x.device, x.dtype, "y")
    st = lib().trellis_f8_silu_mul(_F8_DTYPE[x.dtype], x.data_ptr(), x_row, rows, n, _ptr(q), _ptr(scale), _ptr(y), _stream())
    if st:
        _check(st)
    return (q, scale) if quantize else y


class F8Linear:
    """E4M3 matrices with one f32 scale per 128 x 128 block: w float8_e4m3fn [out, in] and scale
    [ceil(out / 128), ceil(in / 128)], or one per expert, [experts, out, in] and [experts, ...]."""

    def __init__(self, w: torch.Tensor, scale: torch.Tensor):
        _req(w, _E4M3, "w")
        _req(scale, torch.float32, "scale", w.device)
        if w.dim() not in (2, 3):
            raise ValueError(f"w must be [out, in] or [experts, out, in], got {tuple(w.shape)}")
        out, inn = w.shape[-2:]
        want = (*w.shape[:-2], _f8_blocks(out), _f8_blocks(inn))
        if tuple(scale.shape) != want:
            raise ValueError(f"scale must be {want}, got {tuple(scale.shape)}")
        self.w, self.scale, self.device = w, scale, w.device
        self.experts = _i31(w.shape[0], "experts") if w.dim() == 3 else None
        self.in_features, self.out_features = _i31(inn, "in"), _i31(out, "out")
        self._c = CF8Linear(w.data_ptr(), scale.data_ptr(), 1 if self.experts is None else self.experts, inn, out)
        self._ref = ctypes.byref(self._c)


# Workspace sizes of the products by the sizes they follow from (not by tensors).
_f8_nb: Dict[Tuple[int, ...], int] = {}


def _f8_bytes(layer: F8Linear, rows: int) -> int:
    grouped = layer.experts is not None
    key = (layer._c.n_experts, layer.in_features, layer.out_features, rows, grouped, layer.device.index)
    nb = _f8_nb.get(key)
    if nb is None:
        f = lib().trellis_f8_moe_gemm_workspace_bytes if grouped else lib().trellis_f8_gemm_workspace_bytes
        nb = f(layer._ref, rows)
        if nb == 0:
            raise TrellisError(-1, lib().trellis_last_error().decode())
        if len(_f8_nb) >= 4096:
            _f8_nb.clear()
        _f8_nb[key] = nb
    return nb


def trellis_f8_workspace_bytes(layer: F8Linear, rows: int) -> int:
    """Workspace bytes of trellis_f8_gemm (trellis_f8_moe_gemm for experts' matrices)."""
    return _f8_bytes(layer, rows)


def _f8_product(layer: F8Linear, q: torch.Tensor, scale: torch.Tensor, rows: int, dtype, out):
    q_row = _f8_rows(q, "q", _E4M3, layer.device, layer.in_features)
    s_row = _f8_rows(scale, "scale", torch.float32, layer.device, _f8_blocks(layer.in_features))
    if scale.shape[0] != q.shape[0]:
        raise ValueError(f"scale must have one row per row of q ({q.shape[0]}), got {scale.shape[0]}")
    if out is None:
        if dtype not in _F8_DTYPE:
            raise TypeError(f"dtype must be float16 or bfloat16, got {dtype}")
        out = _new2(rows, layer.out_features, dtype, layer.device)
    y_row = _f8_rows(out, "out", None, layer.device, layer.out_features)
    if out.shape[0] != rows:
        raise ValueError(f"out must have {rows} rows, got {out.shape[0]}")
    return q_row, s_row, out, y_row


def trellis_f8_gemm(layer: F8Linear, q: torch.Tensor, scale: torch.Tensor, dtype: torch.dtype = torch.float16,
                    out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M, out] (fp16 or bf16) of E4M3 rows q [M, in] with scales [M, ceil(in / 128)] and one
    matrix; rows of q, scale and ``out`` may have strides of their own."""
    if layer.experts is not None:
        raise ValueError("the layer has one matrix per expert: trellis_f8_moe_gemm takes it")
    M = q.shape[0]
    q_row, s_row, out, y_row = _f8_product(layer, q, scale, M, dtype, out)
    ws = _f8_ws(ws, _f8_bytes(layer, M), layer.device)
    _check(lib().trellis_f8_gemm(layer._ref, q.data_ptr(), q_row, scale.data_ptr(), s_row, M, _F8_DTYPE[out.dtype],
                                 out.data_ptr(), y_row, ws.data_ptr(), ws.numel(), _stream()))
    return out


def trellis_f8_moe_gemm(layer: F8Linear, q: torch.Tensor, scale: torch.Tensor, offsets: torch.Tensor,
                        order: Optional[torch.Tensor] = None, per: int = 1, dtype: torch.dtype = torch.float16,
                        out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows sorted by expert times their experts' matrices: row r in offsets[e] .. offsets[e+1]
    (int32 [experts + 1]) takes matrix e and row r of q, or row order[r] // per of it (``order``
    int32 [rows], trellis_moe_sort's, with per = choices a token).  Rows of ``out`` from the last
    offset on are left alone."""
    if layer.experts is None:
        raise ValueError("the layer has one matrix: trellis_f8_gemm takes it")
    _kv4_int(offsets, "offsets", layer.device)
    if offsets.numel() != layer.experts + 1:
        raise ValueError(f"offsets must have {layer.experts + 1} entries, got {offsets.numel()}")
    if order is not None:
        _kv4_int(order, "order", layer.device)
    rows = q.shape[0] if order is None else _i31(order.numel(), "entries of order")
    q_row, s_row, out, y_row = _f8_product(layer, q, scale, rows, dtype, out)
    ws = _f8_ws(ws, _f8_bytes(layer, rows), layer.device)
    _check(lib().trellis_f8_moe_gemm(layer._ref, q.data_ptr(), q_row, scale.data_ptr(), s_row, q.shape[0], offsets.data_ptr(),
                                     _ptr(order), _i31(per, "per"), rows, _F8_DTYPE[out.dtype], out.data_ptr(), y_row, ws.data_ptr(),
                                     ws.numel(), _stream()))
    return out


def _moe_ids(t: torch.Tensor, name: str, device=None) -> Tuple[int, int]:
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 2 and t.dtype is torch.int32 and t.is_contiguous()
            and t.get_device() == torch._C._cuda_getDevice() and (device is None or t.device == device)
            and not t.numel() >> 31):
        return t.shape
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be [tokens, top]")
    _req(t, torch.int32, name, device)
    if t.device.index != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}: the current device is cuda:{torch._C._cuda_getDevice()}")
    _i31(t.numel(), f"entries of {name}")
    return t.shape[0], t.shape[1]


@functools.lru_cache(maxsize=4096)
def _moe_sort_bytes(tokens: int, top: int, experts: int) -> int:
    _i31(tokens | top | experts, "a size of the sort")
    nb = lib().trellis_moe_sort_workspace_bytes(tokens, top, experts)
    if nb == 0:
        raise TrellisError(-1, lib().trellis_last_error().decode() or f"n_experts={experts} not in 1..2048")
    return nb


@functools.lru_cache(maxsize=None)
def _moe_rows_bytes() -> int:
    return lib().trellis_moe_rows_workspace_bytes()


def trellis_moe_sort(ids: torch.Tensor, n_experts: int, offsets: Optional[torch.Tensor] = None,
                     order: Optional[torch.Tensor] = None, inverse: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Routed ids int32 [tokens, top] (-1: not here) sorted by expert: (offsets [n_experts + 1],
    order [tokens * top]: the entry t * top + j at each position, -1 behind the last, inverse
    [tokens, top]: each entry's position or -1)."""
    tokens, top = _moe_ids(ids, "ids")
    i32, dev = torch.int32, ids.device
    nb = _moe_sort_bytes(tokens, top, n_experts)
    offsets = _out1(offsets, n_experts + 1, dev, i32, "offsets")
    order = _out1(order, tokens * top, dev, i32, "order")
    inverse = _out2(inverse, tokens, top, dev, i32, "inverse")
    ws = _f8_ws(ws, nb, dev)
    _check(lib().trellis_moe_sort(ids.data_ptr(), tokens, top, n_experts, offsets.data_ptr(), order.data_ptr(),
                                  inverse.data_ptr(), ws.data_ptr(), ws.numel(), _stream()))
    return offsets, order, inverse


def trellis_moe_gather(x: torch.Tensor, order: torch.Tensor, per: int, out: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows brought into the experts' order: out[p] = x[order[p] // per], x [tokens, n] of any
    type whose rows are multiples of 4 bytes; rows whose entry is -1 are left as they are.  Its
    gradient is ``trellis_moe_combine(d_out, inverse)``."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    x_row, e = _f8_rows(x, "x", x.dtype), x.element_size()
    _kv4_int(order, "order", x.device)
    tokens, n = x.shape
    rows = _i31(order.numel(), "entries of order")
    out = _out2(out, rows, n, x.device, x.dtype)
    ws = _f8_ws(ws, _moe_rows_bytes(), x.device)
    _check(lib().trellis_moe_gather(x.data_ptr(), x_row * e, tokens, n * e, order.data_ptr(), rows, _i31(per, "per"),
                                    out.data_ptr(), ws.data_ptr(), ws.numel(), _stream()))
    return out


def _moe_weights(weights: Optional[torch.Tensor], inverse: torch.Tensor) -> None:
    if weights is not None:
        _req(weights, torch.float32, "weights", inverse.device)
        if weights.shape != inverse.shape:
            raise ValueError(f"weights must be {tuple(inverse.shape)}, got {tuple(weights.shape)}")


def _moe_rows(t: torch.Tensor, name: str, device, dtype=None, rows=None) -> None:
    """A dense 16-bit [rows, n] tensor."""
    _f8_rows(t, name, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if rows is not None and t.shape[0] != rows:
        raise ValueError(f"{name} must have {rows} rows, got {t.shape[0]}")


def trellis_moe_combine(y: torch.Tensor, inverse: torch.Tensor, weights: Optional[torch.Tensor] = None,
                        add: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                        ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = add[t] + sum_j weights[t, j] * y[inverse[t, j]] over the entries with a position:
    y [rows, n] fp16 or bf16, inverse int32 [tokens, top], weights f32 [tokens, top] (None: ones),
    add [tokens, n] (None: zeros; ``out=add`` adds in place)."""
    tokens, top = _moe_ids(inverse, "inverse")
    _moe_rows(y, "y", inverse.device)
    _moe_weights(weights, inverse)
    n = y.shape[1]
    if add is not None:
        _moe_rows(add, "add", inverse.device, y.dtype, tokens)
        if add.shape[1] != n:
            raise ValueError(f"add must be {(tokens, n)}, got {tuple(add.shape)}")
    out = _out2(out, tokens, n, inverse.device, y.dtype)
    ws = _f8_ws(ws, _moe_rows_bytes(), inverse.device)
    _check(lib().trellis_moe_combine(_F8_DTYPE[y.dtype], y.data_ptr(), y.shape[0], n, inverse.data_ptr(), _ptr(weights), tokens,
                                     top, _ptr(add), out.data_ptr(), ws.data_ptr(), ws.numel(), _stream()))
    return out


def trellis_moe_combine_grad(d_out: torch.Tensor, y: torch.Tensor, inverse: torch.Tensor,
                             weights: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                             d_weights: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """The gradient of trellis_moe_combine: (d_y, d_weights) for d_out [tokens, n] and the forward
    pass's y; rows of d_y (``out``, which may be y) that no entry names are left as they are.
    (That of add is d_out itself.)"""
    tokens, top = _moe_ids(inverse, "inverse")
    _moe_rows(y, "y", inverse.device)
    rows, n = y.shape
    _moe_rows(d_out, "d_out", inverse.device, y.dtype, tokens)
    if d_out.shape[1] != n:
        raise ValueError(f"d_out must be {(tokens, n)}, got {tuple(d_out.shape)}")
    _moe_weights(weights, inverse)
    out = _out2(out, rows, n, inverse.device, y.dtype)
    d_weights = _out2(d_weights, tokens, top, inverse.device, torch.float32, "d_weights")
    ws = _f8_ws(ws, _moe_rows_bytes(), inverse.device)
    _check(lib().trellis_moe_combine_grad(_F8_DTYPE[y.dtype], d_out.data_ptr(), y.data_ptr(), rows, n, inverse.data_ptr(),
                                          _ptr(weights), tokens, top, out.data_ptr(), d_weights.data_ptr(), ws.data_ptr(),
                                          ws.numel(), _stream()))
    return out, d_weights


# ---------------------------------------------------------------------------------------
# Microbenchmarks (include/trellis_micro.h): the machine's ceilings, not the method
# ---------------------------------------------------------------------------------------

MICRO_VALU = {"v_add_u32": 0, "v_mul_lo_u32": 1, "v_mul_u32_u24": 2, "v_mad_u32_u24": 3, "v_mad_u32_u16": 4,
              "v_mul_lo_u16_sdwa": 5, "v_pk_mul_lo_u16": 6, "v_bfe_u32": 7, "v_alignbit_b32": 8,
              "v_perm_b32": 9, "v_bitop3_b32": 10, "v_lshrrev_b32": 11, "v_add_f16_sdwa": 12,
              "v_mul_u32_u24_sdwa": 13, "v_fma_f32": 14}
MICRO_DECODE = {"decode_tile": 100, "decode_tile_mfma": 101, "decode_tile_u24": 102}
MICRO_MFMA = {"f16_16x16x32": (0, 16 * 16 * 32), "f16_32x32x16": (1, 32 * 32 * 16),
              "f8_16x16x128": (2, 16 * 16 * 128), "f8_32x32x64": (3, 32 * 32 * 64)}


def micro_cus() -> int:
    return int(lib().trellis_micro_cus())


def micro_stream_read(buf: torch.Tensor, blocks: int = 0) -> torch.Tensor:
    """Enqueue one stream read of ``buf`` (any dtype, 16-byte aligned, size a multiple of 16)."""
    if not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous GPU tensor")
    nb = buf.numel() * buf.element_size()
    grid = blocks if blocks > 0 else 8 * micro_cus()
    sink = torch.empty(grid * 256, dtype=torch.int32, device=buf.device)
    _check(lib().trellis_micro_stream_read(buf.data_ptr(), nb, blocks, sink.data_ptr(), _stream()))
    return sink


def micro_clock_kernel(kind: str, name: str, iters: int, waves_per_simd: int, device="cuda"):
    """Run one VALU / decode / MFMA micro kernel; returns (cycles, ticks, ms): int64 tensors
    with one entry per workgroup, and the launch's wall time from events (synchronises)."""
    nblk = micro_cus() * waves_per_simd
    cycles = torch.zeros(nblk, dtype=torch.int64, device=device)
    ticks = torch.zeros(nblk, dtype=torch.int64, device=device)
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    if kind == "mfma":
        sink = torch.empty(nblk * 256, dtype=torch.float32, device=device)
        e0.record()
        st = lib().trellis_micro_mfma(MICRO_MFMA[name][0], iters, waves_per_simd, cycles.data_ptr(),
                                      ticks.data_ptr(), sink.data_ptr(), _stream())
    else:
        op = MICRO_VALU.get(name, MICRO_DECODE.get(name))
        sink = torch.empty(nblk * 256, dtype=torch.int32, device=device)
        e0.record()
        st = lib().trellis_micro_valu(op, iters, waves_per_simd, cycles.data_ptr(), ticks.data_ptr(),
                                      sink.data_ptr(), _stream())
    e1.record()
    if st < 0:
        _check(st)
    torch.cuda.synchronize()
    return cycles, ticks, e0.elapsed_time(e1)
