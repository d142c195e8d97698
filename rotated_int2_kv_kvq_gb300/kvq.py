"""Thin Python binding of libkvq.so (include/kvq.h).

Argument marshalling only: every function forwards to the C entry point of the
same name, passing device pointers of torch CUDA tensors and the current CUDA
stream.  Every step of the hot path runs in the library's kernels; there is no
CPU fallback.  If libkvq.so is missing the import fails.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")

KVQ_OK, KVQ_EINVAL, KVQ_ENOSPACE, KVQ_ECUDA, KVQ_ENOTREADY = 0, 1, 2, 3, 4
KVQ_STATUS_BAD_PAGE = 1
KVQ_STATUS_BAD_POS = 2
KVQ_STATUS_BAD_SEQLEN = 4
KVQ_STATUS_BAD_SEQ = 8
KVQ_STATUS_TIMEOUT = 16
KVQ_OUT_ROTATED = 1
KVQ_Q_ROTATED = 2
KVQ_ROPE_HALF, KVQ_ROPE_INTERLEAVED = 0, 1
(KVQ_ROPE_SCALE_NONE, KVQ_ROPE_SCALE_LINEAR, KVQ_ROPE_SCALE_NTK, KVQ_ROPE_SCALE_YARN,
 KVQ_ROPE_SCALE_BANDED) = range(5)
INT2_RECORD_BYTES = 1152
BF16_RECORD_BYTES = 8192

# Every entry point of include/kvq.h, with its ctypes signature.
_P, _I, _SZ, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_LL = ctypes.c_longlong
SIGNATURES = {
    "kvq_create": ([_P, _P], _I),
    "kvq_destroy": ([_P], _I),
    "kvq_page_bytes": ([_P], _SZ),
    "kvq_bf16_page_bytes": ([_P], _SZ),
    "kvq_set_rotation": ([_P, _P, _P, _P], _I),
    "kvq_append": ([_P, _P, _I, _P, _P, _P, _P, _I, _P, _I, _I, _P], _I),
    "kvq_workspace_bytes": ([_P, _I, _I], _SZ),
    "kvq_decode": ([_P, _P, _I, _P, _P, _I, _P, _I, _P, _P, _SZ, _I, _P], _I),
    "kvq_dequant": ([_P, _P, _I, _P, _I, _I, _I, _I, _P, _P, _P], _I),
    "kvq_bf16_append": ([_P, _P, _I, _P, _P, _P, _P, _I, _P, _I, _I, _P], _I),
    "kvq_bf16_workspace_bytes": ([_P, _I, _I], _SZ),
    "kvq_bf16_decode": ([_P, _P, _I, _P, _P, _I, _P, _I, _P, _P, _SZ, _I, _P], _I),
    "kvq_decode_static": ([_P, _P, _I, _P, _P, _I, _P, _I, _P, _I, _P], _I),
    "kvq_optr_workspace_bytes": ([_I, _I, _I, _I, _I], _SZ),
    "kvq_optr_calibrate": ([_I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _F, _F, _F, _F, _I, _F, _P,
                            _P, _P, _SZ, _P], _I),
    "kvq_optr_loss_grad": ([_I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _F, _F, _F, _F, _P, _P, _I,
                            _P, _P, _P, _SZ, _P], _I),
    "kvq_append_decode": ([_P, _P, _I, _P, _P, _P, _P, _I, _P, _I, _P, _P, _SZ, _I, _P], _I),
    "kvq_decode_window": ([_P, _P, _I, _P, _I, _P, _P, _P, _I, _P, _I, _I, _I, _P, _P, _SZ, _I,
                           _P], _I),
    "kvq_append_decode_window": ([_P, _P, _I, _P, _I, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P,
                                  _P, _SZ, _I, _P], _I),
    "kvq_rope_table": ([_P, _I, _I, _P, _P], _I),
    "kvq_rope": ([_P, _P, _LL, _P, _LL, _I, _P, _I, _P, _I, _P], _I),
    "kvq_append_rope": ([_P, _P, _I, _P, _LL, _P, _LL, _P, _P, _I, _P, _I, _I, _P, _P, _P], _I),
    "kvq_bf16_append_rope": ([_P, _P, _I, _P, _LL, _P, _LL, _P, _P, _I, _P, _I, _I, _P, _P, _P],
                             _I),
    "kvq_prefill_workspace_bytes": ([_P, _I, _I], _SZ),
    "kvq_prefill": ([_P, _P, _I, _P, _LL, _P, _I, _P, _I, _P, _I, _P, _P, _SZ, _P], _I),
    "kvq_bf16_prefill_workspace_bytes": ([_P, _I, _I], _SZ),
    "kvq_bf16_prefill": ([_P, _P, _I, _P, _LL, _P, _I, _P, _I, _P, _I, _P, _P, _SZ, _P], _I),
    "kvq_get_status": ([_P, _P, _P], _I),
    "kvq_selftest_wait_timeout": ([_P, _I, _P], _I),
    "kvq_auto_splits": ([_P, _I, _I], _I),
    "kvq_profile_enable": ([_P, _I], _I),
    "kvq_profile_read": ([_P, _P, _P], _I),
    "kvq_strerror": ([_I], ctypes.c_char_p),
}


class KvqLayout(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("group", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("clip_k", ctypes.c_float),
                ("clip_v", ctypes.c_float), ("sm_scale", ctypes.c_float),
                ("flags", ctypes.c_uint32)]


class KvqRopeSpec(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("table_len", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("style", ctypes.c_int32)]


class KvqRopeScaling(ctypes.Structure):
    _fields_ = [("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("orig_len", ctypes.c_double), ("low_turns", ctypes.c_double),
                ("high_turns", ctypes.c_double), ("amplitude", ctypes.c_double),
                ("kind", ctypes.c_int32)]


class KvqError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {code} ({strerror(code)})")
        self.code = code


_lib = None


def load_library():
    """Load libkvq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def strerror(code: int) -> str:
    return load_library().kvq_strerror(int(code)).decode()


def _check(fn, rc):
    if rc != KVQ_OK:
        raise KvqError(fn, rc)


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t, dtypes, name):
    """Device pointer of a contiguous CUDA tensor of one of `dtypes` (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


_BF16 = (torch.bfloat16, torch.int16, torch.uint16) if hasattr(torch, "uint16") else (
    torch.bfloat16, torch.int16)
_U8 = (torch.uint8,)
_I32 = (torch.int32,)
_F32 = (torch.float32,)


class Handle:
    """Owns a kvq_handle*; destroyed with the object."""

    def __init__(self, ptr: int, layout: KvqLayout):
        self.ptr = ctypes.c_void_p(ptr)
        self.layout = layout

    def __del__(self):
        if getattr(self, "ptr", None) and self.ptr.value and _lib is not None:
            _lib.kvq_destroy(self.ptr)
            self.ptr = ctypes.c_void_p(0)

    @property
    def _as_parameter_(self):
        return self.ptr


def make_layout(num_heads, num_kv_heads, clip_k=0.96, clip_v=0.92, sm_scale=0.0,
                out_rotated=False, head_dim=128, group=128, page_size=16,
                q_rotated=False) -> KvqLayout:
    flags = (KVQ_OUT_ROTATED if out_rotated else 0) | (KVQ_Q_ROTATED if q_rotated else 0)
    return KvqLayout(num_heads, num_kv_heads, head_dim, group, page_size, clip_k, clip_v,
                     sm_scale, flags)


# ---- entry points (same names as the C ABI) ------------------------------------

def kvq_create(layout: KvqLayout) -> Handle:
    out = ctypes.c_void_p()
    _check("kvq_create", load_library().kvq_create(ctypes.byref(layout), ctypes.byref(out)))
    h = Handle(out.value, layout)
    h.device = torch.cuda.current_device()
    return h


def kvq_destroy(h: Handle) -> None:
    _check("kvq_destroy", load_library().kvq_destroy(h.ptr))
    h.ptr = ctypes.c_void_p(0)


def kvq_page_bytes(h: Handle) -> int:
    return int(load_library().kvq_page_bytes(h.ptr))


def kvq_bf16_page_bytes(h: Handle) -> int:
    return int(load_library().kvq_bf16_page_bytes(h.ptr))


def kvq_set_rotation(h: Handle, R: torch.Tensor, mu: torch.Tensor, stream=None) -> None:
    _check("kvq_set_rotation", load_library().kvq_set_rotation(
        h.ptr, _ptr(R, _F32, "R"), _ptr(mu, _F32, "mu"), _stream(stream)))


def _append(fn, h, pool, num_pool_pages, K, V, seq_idx, positions, page_table, stream):
    n = int(K.shape[0])
    batch, max_pages = int(page_table.shape[0]), int(page_table.shape[1])
    _check(fn, getattr(load_library(), fn)(
        h.ptr, _ptr(pool, _U8, "pool"), int(num_pool_pages), _ptr(K, _BF16, "K"),
        _ptr(V, _BF16, "V"), _ptr(seq_idx, _I32, "seq_idx"), _ptr(positions, _I32, "positions"),
        n, _ptr(page_table, _I32, "page_table"), batch, max_pages, _stream(stream)))


def kvq_append(h, pool, num_pool_pages, K, V, seq_idx, positions, page_table, stream=None):
    """K, V: [n, Hkv, 128] bf16; seq_idx, positions: int32 [n]; page_table: int32 [B, P]."""
    _append("kvq_append", h, pool, num_pool_pages, K, V, seq_idx, positions, page_table, stream)


def kvq_bf16_append(h, pool, num_pool_pages, K, V, seq_idx, positions, page_table, stream=None):
    _append("kvq_bf16_append", h, pool, num_pool_pages, K, V, seq_idx, positions, page_table,
            stream)


def kvq_workspace_bytes(h: Handle, batch: int, num_splits: int = 0) -> int:
    return int(load_library().kvq_workspace_bytes(h.ptr, int(batch), int(num_splits)))


def kvq_bf16_workspace_bytes(h: Handle, batch: int, num_splits: int = 0) -> int:
    return int(load_library().kvq_bf16_workspace_bytes(h.ptr, int(batch), int(num_splits)))


def kvq_auto_splits(h: Handle, batch: int, max_pages: int) -> int:
    return int(load_library().kvq_auto_splits(h.ptr, int(batch), int(max_pages)))


def _decode(fn, h, pool, num_pool_pages, q, page_table, seq_lens, out, workspace, num_splits,
            stream):
    batch, max_pages = int(page_table.shape[0]), int(page_table.shape[1])
    _check(fn, getattr(load_library(), fn)(
        h.ptr, _ptr(pool, _U8, "pool"), int(num_pool_pages), _ptr(q, _BF16, "q"),
        _ptr(page_table, _I32, "page_table"), max_pages, _ptr(seq_lens, _I32, "seq_lens"),
        batch, _ptr(out, _F32, "out"), _ptr(workspace, _U8, "workspace"),
        int(workspace.numel()), int(num_splits), _stream(stream)))


def kvq_decode(h, pool, num_pool_pages, q, page_table, seq_lens, out, workspace, num_splits=0,
               stream=None):
    """q: [B, H, 128] bf16; out: [B, H, 128] fp32; workspace: uint8, >= kvq_workspace_bytes."""
    _decode("kvq_decode", h, pool, num_pool_pages, q, page_table, seq_lens, out, workspace,
            num_splits, stream)


def kvq_bf16_decode(h, pool, num_pool_pages, q, page_table, seq_lens, out, workspace,
                    num_splits=0, stream=None):
    _decode("kvq_bf16_decode", h, pool, num_pool_pages, q, page_table, seq_lens, out, workspace,
            num_splits, stream)


def kvq_decode_static(h, pool, num_pool_pages, q, page_table, seq_lens, out, num_splits=0,
                      stream=None):
    """kvq_decode with the library's fixed 16 MiB scratch array instead of a
    caller-supplied workspace (for callers that cannot allocate one)."""
    batch, max_pages = int(page_table.shape[0]), int(page_table.shape[1])
    _check("kvq_decode_static", load_library().kvq_decode_static(
        h.ptr, _ptr(pool, _U8, "pool"), int(num_pool_pages), _ptr(q, _BF16, "q"),
        _ptr(page_table, _I32, "page_table"), max_pages, _ptr(seq_lens, _I32, "seq_lens"),
        batch, _ptr(out, _F32, "out"), int(num_splits), _stream(stream)))


def kvq_append_decode(h, pool, num_pool_pages, K_new, V_new, q, page_table, seq_lens, out,
                      workspace, num_splits=0, stream=None):
    """One decode step: append K_new[b], V_new[b] ([B, Hkv, 128] bf16) at
    position seq_lens[b] - 1 of every sequence, then decode (as kvq_decode)."""
    batch, max_pages = int(page_table.shape[0]), int(page_table.shape[1])
    _check("kvq_append_decode", load_library().kvq_append_decode(
        h.ptr, _ptr(pool, _U8, "pool"), int(num_pool_pages), _ptr(K_new, _BF16, "K_new"),
        _ptr(V_new, _BF16, "V_new"), _ptr(q, _BF16, "q"), _ptr(page_table, _I32, "page_table"),
        max_pages, _ptr(seq_lens, _I32, "seq_lens"), batch, _ptr(out, _F32, "out"),
        _ptr(workspace, _U8, "workspace"), int(workspace.numel()), int(num_splits),
        _stream(stream)))


def kvq_decode_window(h, pool, num_pool_pages, bf16_pool, bf16_num_pool_pages, bf16_page_table,
                      q, page_table, seq_lens, sink, recent, out, workspace, num_splits=0,
                      stream=None):
    """Decode with a BF16 window: positions < sink and >= len - recent from the
    BF16 cache (bf16_page_table: int32 [B, P], same shape as page_table), the
    others from the INT2 cache, in one softmax.  Workspace as for kvq_decode."""
    batch, max_pages = int(page_table.shape[0]), int(page_table.shape[1])
    if tuple(bf16_page_table.shape) != (batch, max_pages):
        raise ValueError("bf16_page_table must have the shape of page_table")
    _check("kvq_decode_window", load_library().kvq_decode_window(
        h.ptr, _ptr(pool, _U8, "pool"), int(num_pool_pages), _ptr(bf16_pool, _U8, "bf16_pool"),
        int(bf16_num_pool_pages), _ptr(bf16_page_table, _I32, "bf16_page_table"),
        _ptr(q, _BF16, "q"), _ptr(page_table, _I32, "page_table"), max_pages,
        _ptr(seq_lens, _I32, "seq_lens"), batch, int(sink), int(recent), _ptr(out, _F32, "out"),
        _ptr(workspace, _U8, "workspace"), int(workspace.numel()), int(num_splits),
        _stream(stream)))


def kvq_append_decode_window(h, pool, num_pool_pages, bf16_pool, bf16_num_pool_pages,
                             bf16_page_table, K_new, V_new, q, page_table, seq_lens, sink, recent,
                             out, workspace, num_splits=0, stream=None):
    """One windowed decode step: append K_new[b], V_new[b] ([B, Hkv, 128] bf16) at
    position seq_lens[b] - 1 to the INT2 and the BF16 cache, then decode as
    kvq_decode_window."""
    batch, max_pages = int(page_table.shape[0]), int(page_table.shape[1])
    if tuple(bf16_page_table.shape) != (batch, max_pages):
        raise ValueError("bf16_page_table must have the shape of page_table")
    _check("kvq_append_decode_window", load_library().kvq_append_decode_window(
        h.ptr, _ptr(pool, _U8, "pool"), int(num_pool_pages), _ptr(bf16_pool, _U8, "bf16_pool"),
        int(bf16_num_pool_pages), _ptr(bf16_page_table, _I32, "bf16_page_table"),
        _ptr(K_new, _BF16, "K_new"), _ptr(V_new, _BF16, "V_new"), _ptr(q, _BF16, "q"),
        _ptr(page_table, _I32, "page_table"), max_pages, _ptr(seq_lens, _I32, "seq_lens"), batch,
        int(sink), int(recent), _ptr(out, _F32, "out"), _ptr(workspace, _U8, "workspace"),
        int(workspace.numel()), int(num_splits), _stream(stream)))


# ---- rotary positions ---------------------------------------------------------

_ROPE_STYLES = {"half": KVQ_ROPE_HALF, "interleaved": KVQ_ROPE_INTERLEAVED}
_ROPE_KINDS = {"none": KVQ_ROPE_SCALE_NONE, "linear": KVQ_ROPE_SCALE_LINEAR,
               "ntk": KVQ_ROPE_SCALE_NTK, "yarn": KVQ_ROPE_SCALE_YARN,
               "banded": KVQ_ROPE_SCALE_BANDED}


def make_rope_scaling(kind="none", base=10000.0, factor=1.0, orig_len=0.0, low_turns=1.0,
                      high_turns=None, amplitude=0.0) -> KvqRopeScaling:
    """Frequencies of a table (kvq_rope_scaling).  high_turns defaults to 32 (yarn), 4 (banded)."""
    if high_turns is None:
        high_turns = 32.0 if kind == "yarn" else 4.0
    return KvqRopeScaling(float(base), float(factor), float(orig_len), float(low_turns),
                          float(high_turns), float(amplitude), _ROPE_KINDS[kind])


class Rope:
    """A rotary-position table and how its pairs lie in a head; keeps the table alive."""

    def __init__(self, table: torch.Tensor, style: str):
        if table.dim() != 2:
            raise ValueError("table must be [table_len, rot_dim]")
        self.table, self.style = table, style
        self.spec = KvqRopeSpec(_ptr(table, _F32, "table"), int(table.shape[0]),
                                int(table.shape[1]), _ROPE_STYLES[style])
        self.device = table.get_device()
        self._as_parameter_ = ctypes.byref(self.spec)


def make_rope(table: torch.Tensor, style: str = "half") -> Rope:
    """table: fp32 [table_len, rot_dim] (kvq_rope_table); style: "half" or "interleaved"."""
    return Rope(table, style)


def kvq_rope_table(table: torch.Tensor, scaling: KvqRopeScaling, stream=None) -> None:
    """Fill table (fp32 [table_len, rot_dim]) with cos and sin of every position."""
    if table.dim() != 2:
        raise ValueError("table must be [table_len, rot_dim]")
    p, dev, call = _ptr(table, _F32, "table"), table.get_device(), load_library().kvq_rope_table
    n, rot = table.shape
    if dev == torch.cuda.current_device():
        rc = call(p, n, rot, ctypes.byref(scaling), _raw_stream(stream, dev))
    else:
        with torch.cuda.device(dev):
            rc = call(p, n, rot, ctypes.byref(scaling), _raw_stream(stream, dev))
    _check("kvq_rope_table", rc)


# The calls of a decode step are bound by this module's own time, so the functions
# below look at each tensor once and hand plain integers to ctypes.

def _raw_stream(stream, device: int) -> int:
    """`stream`, or the current stream of the device the tensors are on."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _at(t, dtypes, device, name):
    """Address of a contiguous tensor of one of `dtypes` on CUDA device `device`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the handle on cuda:{device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _vec(t, n, device, name):
    """Address of an int32 [n] tensor."""
    at = _at(t, _I32, device, name)
    if t.dim() != 1 or t.numel() != n:
        raise ValueError(f"{name}: expected [{n}], got {tuple(t.shape)}")
    return at


def _table2(t, device):
    """Address, batch and pages per sequence of a page table."""
    at = _at(t, _I32, device, "page_table")
    if t.dim() != 2:
        raise ValueError(f"page_table: expected [batch, max_pages], got {tuple(t.shape)}")
    batch, max_pages = t.shape
    return at, batch, max_pages


def _rows(t, device, name, heads=None):
    """(address, token stride, n, heads) of bf16 rows [n, heads, 128]; only the tokens may be
    strided."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if t.dtype not in _BF16:
        raise TypeError(f"{name}: dtype {t.dtype} not in {_BF16}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the handle on cuda:{device}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != 128 or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name}: expected [n, {heads or 'heads'}, 128], got {tuple(shape)}")
    n, hh = shape[0], shape[1]
    s0, s1, s2 = t.stride()
    if n and (s2 != 1 or (hh > 1 and s1 != 128)):
        raise ValueError(f"{name}: the heads of a token must be adjacent and contiguous")
    return t.data_ptr(), s0 if n > 1 else hh * 128, n, hh


def _pool(t, pages, page_bytes, device):
    """Address of a pool that holds `pages` pages."""
    at = _at(t, _U8, device, "pool")
    if t.numel() < pages * page_bytes:
        raise ValueError(f"pool: {t.numel()} bytes hold fewer than {pages} pages")
    return at


def _rope_on(rope, device):
    if rope.device != device:
        raise ValueError(f"the rotary-position table is on cuda:{rope.device}, the handle on "
                         f"cuda:{device}")
    return rope


def kvq_rope(h, x, y, positions, rope: Rope, inverse=False, stream=None):
    """y = x rotated by positions; x, y: bf16 [n, heads, 128] (tokens may be strided), y may be x;
    positions: int32 [n]."""
    dev = h.device
    px, sx, n, heads = _rows(x, dev, "x")
    py, sy, ny, hy = _rows(y, dev, "y")
    if ny != n or hy != heads:
        raise ValueError("y must have the shape of x")
    _check("kvq_rope", load_library().kvq_rope(
        h.ptr, px, sx, py, sy, heads, _vec(positions, n, dev, "positions"), n, _rope_on(rope, dev),
        1 if inverse else 0, _raw_stream(stream, dev)))


def _append_rope(int2, h, pool, num_pool_pages, K, V, seq_idx, positions, page_table, rope,
                 rope_positions, stream):
    dev, hkv = h.device, h.layout.num_kv_heads
    pk, sk, n, _ = _rows(K, dev, "K", hkv)
    pv, sv, nv, _ = _rows(V, dev, "V", hkv)
    if nv != n:
        raise ValueError("K and V must have the same number of tokens")
    pt, batch, max_pages = _table2(page_table, dev)
    pages, record = int(num_pool_pages), INT2_RECORD_BYTES if int2 else BF16_RECORD_BYTES
    fn = "kvq_append_rope" if int2 else "kvq_bf16_append_rope"
    _check(fn, getattr(load_library(), fn)(
        h.ptr, _pool(pool, pages, hkv * record, dev), pages, pk, sk, pv, sv,
        _vec(seq_idx, n, dev, "seq_idx"), _vec(positions, n, dev, "positions"), n, pt, batch,
        max_pages, _rope_on(rope, dev),
        None if rope_positions is None else _vec(rope_positions, n, dev, "rope_positions"),
        _raw_stream(stream, dev)))


def kvq_append_rope(h, pool, num_pool_pages, K, V, seq_idx, positions, page_table, rope: Rope,
                    rope_positions=None, stream=None):
    """kvq_append with the keys rotated on the way.  K, V: bf16 [n, Hkv, 128], tokens may be
    strided (slices of a fused projection); rope_positions: int32 [n] if the angles' positions
    are not the cache's."""
    _append_rope(True, h, pool, num_pool_pages, K, V, seq_idx, positions, page_table,
                 rope, rope_positions, stream)


def kvq_bf16_append_rope(h, pool, num_pool_pages, K, V, seq_idx, positions, page_table,
                         rope: Rope, rope_positions=None, stream=None):
    """kvq_bf16_append with the keys rotated on the way (arguments as kvq_append_rope)."""
    _append_rope(False, h, pool, num_pool_pages, K, V, seq_idx, positions,
                 page_table, rope, rope_positions, stream)


# ---- attention of a chunk of new tokens -----------------------------------------

def kvq_prefill_workspace_bytes(h: Handle, batch: int, n: int) -> int:
    return int(load_library().kvq_prefill_workspace_bytes(h.ptr, int(batch), int(n)))


def kvq_bf16_prefill_workspace_bytes(h: Handle, batch: int, n: int) -> int:
    return int(load_library().kvq_bf16_prefill_workspace_bytes(h.ptr, int(batch), int(n)))


def _prefill(int2, h, pool, num_pool_pages, q, cu_q, page_table, seq_lens, out, workspace, stream):
    dev, H = h.device, h.layout.num_heads
    pq, sq, n, _ = _rows(q, dev, "q", H)
    pt, batch, max_pages = _table2(page_table, dev)
    po = _at(out, _BF16, dev, "out")
    if tuple(out.shape) != (n, H, 128):
        raise ValueError(f"out: expected [{n}, {H}, 128], got {tuple(out.shape)}")
    pages, record = int(num_pool_pages), INT2_RECORD_BYTES if int2 else BF16_RECORD_BYTES
    fn = "kvq_prefill" if int2 else "kvq_bf16_prefill"
    _check(fn, getattr(load_library(), fn)(
        h.ptr, _pool(pool, pages, h.layout.num_kv_heads * record, dev), pages, pq, sq,
        _vec(cu_q, batch + 1, dev, "cu_q"), n, pt, max_pages,
        _vec(seq_lens, batch, dev, "seq_lens"), batch, po, _at(workspace, _U8, dev, "workspace"),
        workspace.numel(), _raw_stream(stream, dev)))


def kvq_prefill(h, pool, num_pool_pages, q, cu_q, page_table, seq_lens, out, workspace,
                stream=None):
    """Causal attention of each sequence's new tokens over its INT2 cache.  q: bf16 [n, H, 128]
    (tokens may be strided); cu_q: int32 [B + 1], sequence b's rows are cu_q[b]:cu_q[b + 1], the
    last of its seq_lens[b] positions; out: bf16 [n, H, 128]; workspace: uint8,
    >= kvq_prefill_workspace_bytes(h, B, n)."""
    _prefill(True, h, pool, num_pool_pages, q, cu_q, page_table, seq_lens, out, workspace, stream)


def kvq_bf16_prefill(h, pool, num_pool_pages, q, cu_q, page_table, seq_lens, out, workspace,
                     stream=None):
    """kvq_prefill over the BF16 cache (workspace: kvq_bf16_prefill_workspace_bytes)."""
    _prefill(False, h, pool, num_pool_pages, q, cu_q, page_table, seq_lens, out, workspace, stream)


def kvq_dequant(h, pool, num_pool_pages, page_table, seq, start, length, K_out=None, V_out=None,
                stream=None):
    _check("kvq_dequant", load_library().kvq_dequant(
        h.ptr, _ptr(pool, _U8, "pool"), int(num_pool_pages), _ptr(page_table, _I32, "page_table"),
        int(page_table.shape[1]), int(seq), int(start), int(length), _ptr(K_out, _F32, "K_out"),
        _ptr(V_out, _F32, "V_out"), _stream(stream)))


def kvq_get_status(h: Handle, stream=None) -> int:
    bits = ctypes.c_uint32()
    _check("kvq_get_status", load_library().kvq_get_status(h.ptr, ctypes.byref(bits),
                                                           _stream(stream)))
    return int(bits.value)


def kvq_selftest_wait_timeout(h: Handle, limit_us: int, stream=None) -> None:
    _check("kvq_selftest_wait_timeout",
           load_library().kvq_selftest_wait_timeout(h.ptr, int(limit_us), _stream(stream)))


def kvq_profile_enable(h: Handle, enable: bool = True) -> None:
    _check("kvq_profile_enable", load_library().kvq_profile_enable(h.ptr, 1 if enable else 0))


def kvq_profile_read(h: Handle):
    """(total milliseconds of the split-K attention kernel, launches) since enable."""
    ms = ctypes.c_double()
    n = ctypes.c_int()
    _check("kvq_profile_read", load_library().kvq_profile_read(h.ptr, ctypes.byref(ms),
                                                               ctypes.byref(n)))
    return float(ms.value), int(n.value)


def kvq_optr_workspace_bytes(num_kv_heads, T, Nq, G, Dm) -> int:
    return int(load_library().kvq_optr_workspace_bytes(int(num_kv_heads), int(T), int(Nq), int(G),
                                                       int(Dm)))


def kvq_optr_calibrate(K, V, Q, W_O, R0, mu, clip_k, clip_v, lambda_k=1.0, lr=1e-3, steps=80,
                       sm_scale=0.0, workspace=None, stream=None):
    """OptR calibration of the key and value rotations of every KV head.
    K, V: bf16 [Hkv, T, 128]; Q: bf16 [Hkv, Nq, G, 128]; W_O: fp32 [Hkv, Dm, G*128];
    R0: fp32 [2, Hkv, 128, 128]; mu: fp32 [Hkv, 128].  Returns (R fp32
    [2, Hkv, 128, 128], history fp32 [2, steps + 1, Hkv]) as CUDA tensors."""
    Hkv, T = int(K.shape[0]), int(K.shape[1])
    Nq, G, Dm = int(Q.shape[1]), int(Q.shape[2]), int(W_O.shape[1])
    R = torch.empty((2, Hkv, 128, 128), dtype=torch.float32, device=K.device)
    hist = torch.empty((2, int(steps) + 1, Hkv), dtype=torch.float32, device=K.device)
    if workspace is None:
        workspace = torch.empty(kvq_optr_workspace_bytes(Hkv, T, Nq, G, Dm), dtype=torch.uint8,
                                device=K.device)
    _check("kvq_optr_calibrate", load_library().kvq_optr_calibrate(
        Hkv, T, Nq, G, Dm, _ptr(K, _BF16, "K"), _ptr(V, _BF16, "V"), _ptr(Q, _BF16, "Q"),
        _ptr(W_O, _F32, "W_O"), _ptr(R0, _F32, "R0"), _ptr(mu, _F32, "mu"), float(clip_k),
        float(clip_v), float(lambda_k), float(lr), int(steps), float(sm_scale), _ptr(R, _F32, "R"),
        _ptr(hist, _F32, "history"), _ptr(workspace, _U8, "workspace"), int(workspace.numel()),
        _stream(stream)))
    return R, hist


def kvq_optr_loss_grad(K, V, Q, W_O, R0, mu, clip_k, clip_v, A_key, A_value=None, which=0,
                       lambda_k=1.0, sm_scale=0.0, workspace=None, stream=None):
    """Loss [Hkv] and d loss / dA [Hkv, 128, 128] of the key (which = 0) or value
    (which = 1) calibration objective, as CUDA tensors."""
    Hkv, T = int(K.shape[0]), int(K.shape[1])
    Nq, G, Dm = int(Q.shape[1]), int(Q.shape[2]), int(W_O.shape[1])
    loss = torch.empty(Hkv, dtype=torch.float32, device=K.device)
    grad = torch.empty((Hkv, 128, 128), dtype=torch.float32, device=K.device)
    if workspace is None:
        workspace = torch.empty(kvq_optr_workspace_bytes(Hkv, T, Nq, G, Dm), dtype=torch.uint8,
                                device=K.device)
    _check("kvq_optr_loss_grad", load_library().kvq_optr_loss_grad(
        Hkv, T, Nq, G, Dm, _ptr(K, _BF16, "K"), _ptr(V, _BF16, "V"), _ptr(Q, _BF16, "Q"),
        _ptr(W_O, _F32, "W_O"), _ptr(R0, _F32, "R0"), _ptr(mu, _F32, "mu"), float(clip_k),
        float(clip_v), float(lambda_k), float(sm_scale), _ptr(A_key, _F32, "A_key"),
        _ptr(A_value, _F32, "A_value"), int(which), _ptr(loss, _F32, "loss"),
        _ptr(grad, _F32, "grad"), _ptr(workspace, _U8, "workspace"), int(workspace.numel()),
        _stream(stream)))
    return loss, grad


def kvq_strerror(code: int) -> str:
    return strerror(code)
