"""GB300-native paged GQA attention: Python binding of ``libpagedattn.so``.

Thin ctypes marshalling over the C ABI in ``include/pagedattn.h``, with a compiled fast path for the
calls of a serving step (``csrc/fastcall.cpp``): every computation runs in the library's CUDA
kernels. PyTorch only provides device memory and streams. There is no CPU
or fallback path: if the shared library has not been built, ``load()`` raises.

Calls (same names as the C ABI):

* ``kv_append_paged``   write new tokens' K/V rows into their page slots
* ``attn_decode_paged`` one decode step over a paged KV cache (split-KV + log-sum-exp merge)
* ``attn_prefill_chunk`` causal attention of query chunks over their cached prefix + themselves
* ``attn_merge_lse``    combine partial results over disjoint key sets
* ``paged_step_plan``   block tables, positions and slot maps of a step from request lengths
* ``paged_release``     give pages of finished or windowed requests back to the free list
* ``rope_append_paged`` rotary positions of new q and k rows, K/V written into their slots
* ``attn_decode_paged_shared`` a decode step of rows that share leading pages, read once a group
* ``beam_select``       the best continuations of each request's beams, over beams and vocabulary
* ``paged_fork``        block tables follow the beams: pages shared, copied, given back
* ``paged_copy_pages``  the page copies that a fork orders, in all layers' pools
"""
from __future__ import annotations

import collections
import ctypes
import importlib.util
import os

import torch

__all__ = [
    "load", "PagedAttnError", "Dims", "DEFAULT_DIMS",
    "kv_append_paged", "attn_decode_paged", "attn_decode_paged_noalloc", "attn_prefill_chunk",
    "attn_merge_lse", "adaptor_mlp_merge4", "adaptor_workspace_size", "LaunchOpts",
    "decode_workspace_size", "decode_kernels_per_call", "prefill_workspace_size",
    "prefill_score_workspace_size",
    "read_device_status", "debug_decode_starve",
    "paged_step_plan", "StepPlan", "paged_release", "rope_append_paged", "rope_inv_freq",
    "RopeScaling", "ScoreOpts",
    "attn_decode_paged_shared", "decode_shared_workspace_size", "beam_select", "BeamStep",
    "beam_workspace_size", "paged_fork", "ForkPlan", "fork_workspace_size", "paged_copy_pages",
    "DEV_ERR_PAGE_OOB", "DEV_ERR_LENGTH", "DEV_ERR_TIMEOUT", "DEV_ERR_INTERNAL",
    "DEV_ERR_NO_PAGES", "lib_path",
]

DEV_ERR_PAGE_OOB = 1
DEV_ERR_LENGTH = 2
DEV_ERR_TIMEOUT = 4
DEV_ERR_INTERNAL = 8
DEV_ERR_NO_PAGES = 16

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None
_FAST = None  # the fast path's module (csrc/fastcall.cpp), once the library is loaded and if it is there


def lib_path() -> str:
    return os.path.join(_HERE, "_lib", "libpagedattn.so")


class Dims(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32)]


DEFAULT_DIMS = (16, 8, 128, 16)


class PagedAttnError(RuntimeError):
    def __init__(self, call: str, code: int):
        lib = load()
        text = lib.pa_status_string(code).decode()
        detail = lib.pa_last_error().decode()
        super().__init__(f"{call} failed: {text} ({code}){': ' + detail if detail else ''}")
        self.code = code


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float

class LaunchOpts(ctypes.Structure):
    """pa_launch_opts: max_ctas > 0 caps a call's persistent grid (0 = one CTA per SM)."""
    _fields_ = [("max_ctas", ctypes.c_int32)]


class ScoreOpts(ctypes.Structure):
    """pa_score_opts (device pointers as integers)."""
    _fields_ = [("softcap", ctypes.c_float), ("alibi_slopes", ctypes.c_void_p),
                ("window", ctypes.c_int32), ("prefix_lens", ctypes.c_void_p),
                ("max_prefix_len", ctypes.c_int32), ("row_start", ctypes.c_void_p)]


class RopeScaling(ctypes.Structure):
    """pa_rope_scaling."""
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double),
                ("original_max_position", ctypes.c_double),
                ("low_freq_factor", ctypes.c_double), ("high_freq_factor", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("attn_factor", ctypes.c_double)]


def _opts(max_ctas):
    if max_ctas is None:
        return None, None
    m = int(max_ctas)
    if m < 0:
        raise ValueError("max_ctas must be >= 0")
    o = LaunchOpts(m)
    return o, ctypes.byref(o)


_SIGS = {
    "kv_append_paged": (_I32, [Dims, _P, _P, _I32, _P, _P, _I32, _P, _I32, _P, _P, _I64, _P, _P]),
    "pa_decode_workspace_size": (_SZ, [Dims, _I32, _I32, _I32]),
    "pa_decode_kernels_per_call": (_I32, [Dims, _I32, _I32, _I32]),
    "attn_decode_paged": (_I32, [Dims, _P, _P, _P, _I64, _P, _I32, _P, _I32, _I32, _F, _I32, _P, _P,
                                 _P, _SZ, _P, _P]),
    "pa_debug_decode_starve": (_I32, [_I32]),
    "attn_decode_paged_noalloc": (_I32, [Dims, _P, _P, _P, _I64, _P, _I32, _P, _I32, _I32, _F, _P,
                                         _P, _P, _P]),
    "pa_prefill_workspace_size": (_SZ, [Dims, _I32, _I32, _I32]),
    "attn_prefill_chunk": (_I32, [Dims, _P, _P, _I32, _P, _P, _I64, _P, _I32, _P, _I32, _I32, _I32,
                                  _F, _P, _P, _P, _SZ, _P, _P]),
    "attn_decode_paged_ex": (_I32, [Dims, _P, _P, _P, _I64, _P, _I32, _P, _I32, _I32, _F, _I32, _P,
                                    _P, _P, _SZ, _P, _P, _P]),
    "attn_prefill_chunk_ex": (_I32, [Dims, _P, _P, _I32, _P, _P, _I64, _P, _I32, _P, _I32, _I32,
                                     _I32, _F, _P, _P, _P, _SZ, _P, _P, _P]),
    "attn_decode_paged_score": (_I32, [Dims, _P, _P, _P, _I64, _P, _I32, _P, _I32, _I32, _F, _I32,
                                       _P, _P, _P, _SZ, _P, _P, _P, ctypes.POINTER(ScoreOpts)]),
    "pa_prefill_score_workspace_size": (_SZ, [Dims, _I32, _I32]),
    "attn_prefill_chunk_score": (_I32, [Dims, _P, _P, _I32, _P, _P, _I64, _P, _I32, _P, _I32, _I32,
                                        _I32, _F, _P, _P, _P, _SZ, _P, _P, _P,
                                        ctypes.POINTER(ScoreOpts)]),
    "attn_merge_lse": (_I32, [_I32, _I32, _I32, _I32, _P, _P, _P, _P, _P]),
    "pa_adaptor_workspace_size": (_SZ, [_I32]),
    "adaptor_mlp_merge4": (_I32, [_I32, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _SZ, _P, _P]),
    "paged_step_plan": (_I32, [_P, _P, _I32, _P, _I32, _P, _I32, _P, _I64, _I32, _P, _P, _P, _P, _P,
                               _P, _P]),
    "paged_release": (_I32, [_P, _P, _I32, _P, _I32, _P, _I32, _P, _I64, _P, _P, _P]),
    "pa_rope_inv_freq": (_I32, [_I32, ctypes.c_double, ctypes.POINTER(RopeScaling), _P,
                                ctypes.POINTER(_F)]),
    "rope_append_paged": (_I32, [Dims, _I32, _I32, _P, _F, _P, _I64, _P, _I64, _P, _I64, _I32, _P,
                                 _P, _P, _P, _F, _P, _P, _P, _I64, _P, _P]),
    "pa_decode_shared_workspace_size": (_SZ, [Dims, _I32, _I32, _I32]),
    "attn_decode_paged_shared": (_I32, [Dims, _P, _P, _P, _I64, _P, _I32, _P, _I32, _P, _P, _I32, _I32,
                                        _I32, _F, _P, _P, _P, _SZ, _P, _P]),
    "pa_beam_workspace_size": (_SZ, [_I32, _I32, _I32, _I32]),
    "beam_select": (_I32, [_P, _I32, _I64, _I32, _I32, _I32, _P, _P, _I32, _I32, _P, _P, _P, _P, _P,
                           _SZ, _P]),
    "pa_fork_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "paged_fork": (_I32, [_P, _P, _I32, _I32, _P, _I32, _P, _I32, _P, _I64, _P, _P, _P, _P, _P, _SZ, _P,
                          _P]),
    "paged_copy_pages": (_I32, [Dims, _P, _I32, ctypes.POINTER(_P), _I32, _I64, _P, _P]),
    "pa_read_device_status": (_I32, [_P, ctypes.POINTER(ctypes.c_uint32), _P]),
    "pa_status_string": (ctypes.c_char_p, [_I32]),
    "pa_last_error": (ctypes.c_char_p, []),
    "pa_version": (_I32, []),
}


def load():
    """Load the built library (raises if it is missing: there is no fallback)."""
    global _LIB, _FAST
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
        _FAST = _load_fast()
    return _LIB


def _load_fast():
    """The fast path, if it was built for this PyTorch; None otherwise."""
    path = os.path.join(_HERE, "_lib", "_pa_call.so")
    if not os.path.exists(path):
        return None
    try:
        spec = importlib.util.spec_from_file_location("_pa_call", path)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
    except ImportError:
        return None
    if mod.torch_version.split("+")[0] != torch.__version__.split("+")[0]:
        return None
    mod.set_error(PagedAttnError)
    return mod


# ----------------------------------------------------------------------------------------------
# marshalling helpers
# ----------------------------------------------------------------------------------------------
_dims_cache = {}


def _dims(dims):
    """The Dims of a (num_q_heads, num_kv_heads, head_dim, page_size) tuple, made once per tuple."""
    dims = DEFAULT_DIMS if dims is None else dims
    try:
        return _dims_cache[dims]
    except (KeyError, TypeError):
        d = Dims(*(dims or DEFAULT_DIMS))
        if isinstance(dims, tuple):
            _dims_cache[dims] = d
        return d


def _ptr(t):
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    """The stream's handle; the current stream of the current device for None (read directly: making
    a torch.cuda.Stream object for it takes longer than a kernel launch)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _empty(shape, dtype, device, stream):
    """A new tensor for work on `stream` (None: the current one): allocated from that stream's
    memory, so that the block is neither still read by other work nor handed out again before this
    work ran."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):  # (any object that has a stream's handle will do)
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _need(t, name, dtype, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _handle(stream):
    """A stream's handle for the fast path (None: the current stream)."""
    return None if stream is None else stream.cuda_stream


def _attn_outputs(q, out, lse, want_lse, stream):
    """out and lse of an attention call, new ones where they were not given (and q has a shape)."""
    if isinstance(q, torch.Tensor) and q.is_cuda and q.dim() == 3:
        if out is None:
            out = _empty(q.shape, torch.bfloat16, q.device, stream)
        if lse is None and want_lse:
            lse = _empty(q.shape[:2], torch.float32, q.device, stream)
    return out, lse


def _check(call, code):
    if code != 0:
        raise PagedAttnError(call, code)


def _on_device(call, *tensors):
    """Every tensor must live on the current CUDA device: the library launches there, and a
    pointer into another GPU's memory would be read by the wrong device."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.device.index != dev:
            raise ValueError(f"{call}: tensors must be on the current CUDA device (cuda:{dev}), "
                             f"got {t.device}")


def _shape(name, t, shape):
    """t must have this shape (None entries match anything)."""
    if t.dim() != len(shape) or any(w is not None and d != w for d, w in zip(t.shape, shape)):
        raise ValueError(f"{name} must have shape {tuple('*' if w is None else w for w in shape)}, "
                         f"got {tuple(t.shape)}")


def _rows_at_least(name, t, n):
    if t.shape[0] < n:
        raise ValueError(f"{name} must have at least {n} rows, got {t.shape[0]}")


_heads_cache = {}


def _heads(dims):
    """(query heads, KV heads) of a shape the library supports, else None: the library itself
    then rejects the call (PA_ERR_UNSUPPORTED) and the shape checks below are skipped."""
    dims = DEFAULT_DIMS if dims is None else dims
    try:
        return _heads_cache[dims]
    except (KeyError, TypeError):
        pass
    d = _dims(dims)
    r = None
    if (d.head_dim == 128 and d.page_size == 16 and d.num_kv_heads in (1, 2, 4, 8)
            and d.num_q_heads == 2 * d.num_kv_heads):
        r = d.num_q_heads, d.num_kv_heads
    if isinstance(dims, tuple):
        _heads_cache[dims] = r
    return r


def _tensor(call, t, name, dtype, dev):
    """data_ptr of a contiguous tensor of this type on device `dev`: the checks of _need and
    _on_device in the fewest attribute reads, since a small call's time is its checks'."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name} must be a tensor") from None
    _need(t, name, dtype)
    _on_device(call, t)
    raise ValueError(f"{call}: tensors must be on one device (cuda:{dev}), got {t.device}")


def _device(call, t, name, dtype):
    """The CUDA device index of a call's first tensor, which has to be the current device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _need(t, name, dtype)
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        _on_device(call, t)
    return dev


def _need_dims(*named):
    """Every (name, tensor, dims) must have that many dims."""
    for name, t, d in named:
        if t.dim() != d:
            raise ValueError(f"{name} must have {d} dims, got {t.dim()}")


def _sized(name, t, shape):
    """t must have exactly this shape."""
    if t.shape != shape:
        _shape(name, t, shape)


def _pools(k_pool, v_pool, hkv):
    _shape("k_pool", k_pool, (None, 16, hkv, 128))
    _shape("v_pool", v_pool, tuple(k_pool.shape))


def _given(t, name, dtype, shape):
    """A caller-provided output buffer: dtype, layout and shape checked, since the kernels write
    every element of it."""
    if t is not None:
        _need(t, name, dtype)
        _shape(name, t, shape)


# ----------------------------------------------------------------------------------------------
# the four calls
# ----------------------------------------------------------------------------------------------
def kv_append_paged(k_new, v_new, cu_new_lens, start_pos, block_table, k_pool, v_pool, *,
                    status=None, stream=None, dims=None):
    """Write rows of k_new/v_new [T, Hkv, D] into the pools at their block-table slots."""
    for t, n, d in ((k_new, "k_new", torch.bfloat16), (v_new, "v_new", torch.bfloat16),
                    (cu_new_lens, "cu_new_lens", torch.int32), (start_pos, "start_pos", torch.int32),
                    (block_table, "block_table", torch.int32), (k_pool, "k_pool", torch.bfloat16),
                    (v_pool, "v_pool", torch.bfloat16)):
        _need(t, n, d)
    B = start_pos.shape[0]
    _rows_at_least("cu_new_lens", cu_new_lens, B + 1)
    _rows_at_least("block_table", block_table, B)
    heads = _heads(dims)
    if heads is not None:
        _shape("k_new", k_new, (None, heads[1], 128))
        _shape("v_new", v_new, tuple(k_new.shape))
        _pools(k_pool, v_pool, heads[1])
    if status is not None:
        _need(status, "status", torch.int32)
    _on_device("kv_append_paged", k_new, v_new, cu_new_lens, start_pos, block_table, k_pool,
               v_pool, status)
    lib = load()
    _check("kv_append_paged", lib.kv_append_paged(
        _dims(dims), _ptr(k_new), _ptr(v_new), k_new.shape[0], _ptr(cu_new_lens), _ptr(start_pos),
        start_pos.shape[0], _ptr(block_table), block_table.shape[1], _ptr(k_pool), _ptr(v_pool),
        k_pool.shape[0], _ptr(status), _stream(stream)))


def decode_workspace_size(batch: int, max_seq_len: int, split_tokens: int = 0, dims=None) -> int:
    return int(load().pa_decode_workspace_size(_dims(dims), batch, max_seq_len, split_tokens))


def decode_kernels_per_call(batch: int, max_seq_len: int, split_tokens: int = 0, dims=None) -> int:
    """Kernels one attn_decode_paged call launches (1: single-launch short-batch path, 2: split
    kernel + merge; 0 for an empty or unsupported call)."""
    return int(load().pa_decode_kernels_per_call(_dims(dims), batch, max_seq_len, split_tokens))


def prefill_workspace_size(batch: int, max_q_len: int, max_seq_len: int, dims=None) -> int:
    return int(load().pa_prefill_workspace_size(_dims(dims), batch, max_q_len, max_seq_len))


def prefill_score_workspace_size(batch: int, total_q: int, dims=None) -> int:
    """Workspace of attn_prefill_chunk with score options."""
    return int(load().pa_prefill_score_workspace_size(_dims(dims), batch, total_q))


_ws_sizes = {}


def _workspace_size(fn, *key):
    """fn(*key), a size that depends on the arguments and the device alone, looked up once."""
    if isinstance(key[-1], list):  # dims given as a list
        key = key[:-1] + (tuple(key[-1]),)
    key = (fn, torch.cuda.current_device()) + key
    n = _ws_sizes.get(key)
    if n is None:
        if len(_ws_sizes) > 4096:  # a server's shapes are few; this bounds a caller that varies them
            _ws_sizes.clear()
        n = _ws_sizes[key] = fn(*key[2:])
    return n


def _workspace(nbytes, device, workspace, stream=None):
    if workspace is not None:
        return workspace
    return _empty(max(nbytes, 256), torch.uint8, device, stream)


def _score(call, dev, hq, batch, rows, max_seq_len, softcap, alibi_slopes, window, prefix_lens,
           max_prefix_len, row_start):
    """The score options as a ScoreOpts, or None when none is set. Tensors are checked here; the
    caller keeps them alive until the call has been made."""
    slopes = prefix = start = 0
    if alibi_slopes is not None:
        slopes = _tensor(call, alibi_slopes, "alibi_slopes", torch.float32, dev)
        _sized("alibi_slopes", alibi_slopes, (hq,))
    if prefix_lens is not None:
        prefix = _tensor(call, prefix_lens, "prefix_lens", torch.int32, dev)
        _rows_at_least("prefix_lens", prefix_lens, batch)
        if max_prefix_len is None:
            max_prefix_len = max_seq_len
    else:
        max_prefix_len = 0
    if row_start is not None:
        start = _tensor(call, row_start, "row_start", torch.int32, dev)
        _rows_at_least("row_start", row_start, rows)
    elif not softcap and not window and not slopes and prefix_lens is None:
        return None
    return ScoreOpts(float(softcap), slopes, int(window), prefix, int(max_prefix_len), start)


def attn_decode_paged(q, k_pool, v_pool, block_table, seq_lens, max_seq_len: int,
                      softmax_scale: float, *, split_tokens: int = 0, out=None, lse=None,
                      workspace=None, status=None, stream=None, want_lse=True, dims=None,
                      max_ctas=None, softcap: float = 0.0, alibi_slopes=None, window: int = 0,
                      prefix_lens=None, max_prefix_len=None, row_start=None):
    """Decode attention: q [B, Hq, D] over each sequence's cached keys. Returns (out, lse).

    split_tokens: keys per split-KV range (whole pages); 0 = one equal share per SM.
    max_ctas: cap on the persistent grid (attn_decode_paged_ex); None = the plain call.

    Score options (attn_decode_paged_score). Key j is seen from position i when j < prefix_lens[b]
    or max(row_start[b], i - window + 1) <= j <= i; its score is softcap * tanh(s / softcap) minus
    alibi_slopes[h] * |i - j|. max_prefix_len: host bound of prefix_lens (default max_seq_len)."""
    call = "attn_decode_paged"
    if _FAST is not None:
        o, l = _attn_outputs(q, out, lse, want_lse, stream)
        if _FAST.decode(q, k_pool, v_pool, block_table, seq_lens, max_seq_len, softmax_scale,
                        split_tokens, o, l, workspace, status, _handle(stream), dims, max_ctas, softcap,
                        alibi_slopes, window, prefix_lens, max_prefix_len, row_start):
            return o, l
    dev = _device(call, q, "q", torch.bfloat16)
    pq = _tensor(call, q, "q", torch.bfloat16, dev)
    pk = _tensor(call, k_pool, "k_pool", torch.bfloat16, dev)
    pv = _tensor(call, v_pool, "v_pool", torch.bfloat16, dev)
    pbt = _tensor(call, block_table, "block_table", torch.int32, dev)
    psl = _tensor(call, seq_lens, "seq_lens", torch.int32, dev)
    if not (q.dim() == 3 and k_pool.dim() == v_pool.dim() == 4 and block_table.dim() == 2
            and seq_lens.dim() == 1):
        _need_dims(("q", q, 3), ("k_pool", k_pool, 4), ("v_pool", v_pool, 4),
                   ("block_table", block_table, 2), ("seq_lens", seq_lens, 1))
    B, hq, _ = q.shape
    rows, bt_stride = block_table.shape
    if rows < B:
        _rows_at_least("block_table", block_table, B)
    _rows_at_least("seq_lens", seq_lens, B)
    num_pages = k_pool.shape[0]
    heads = _heads(dims)
    if heads is not None:
        _sized("q", q, (B, heads[0], 128))
        pool = (num_pages, 16, heads[1], 128)
        _sized("k_pool", k_pool, pool)
        _sized("v_pool", v_pool, pool)
    if out is None:
        out = _empty(q.shape, torch.bfloat16, q.device, stream)
        po = out.data_ptr()
    else:
        po = _tensor(call, out, "out", torch.bfloat16, dev)
        _sized("out", out, q.shape)
    if lse is None:
        if want_lse:
            lse = _empty((B, hq), torch.float32, q.device, stream)
        pl = None if lse is None else lse.data_ptr()
    else:
        pl = _tensor(call, lse, "lse", torch.float32, dev)
        _sized("lse", lse, (B, hq))
    max_seq_len, split_tokens = int(max_seq_len), int(split_tokens)
    score = _score(call, dev, hq, B, B, max_seq_len, softcap, alibi_slopes, window, prefix_lens,
                   max_prefix_len, row_start)
    if workspace is None:
        nbytes = _workspace_size(decode_workspace_size, B, max_seq_len, split_tokens, dims)
        workspace = _workspace(nbytes, q.device, None, stream)
    else:
        _on_device(call, workspace)
    ps = None if status is None else _tensor(call, status, "status", torch.int32, dev)
    lib = load()
    args = (_dims(dims), pq, pk, pv, num_pages, pbt, bt_stride, psl, B, max_seq_len,
            float(softmax_scale), split_tokens, po, pl, workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), ps, _stream(stream))
    keep, ref = _opts(max_ctas)
    if score is not None:
        _check("attn_decode_paged_score",
               lib.attn_decode_paged_score(*args, ref, ctypes.byref(score)))
    elif ref is None:
        _check(call, lib.attn_decode_paged(*args))
    else:
        _check("attn_decode_paged_ex", lib.attn_decode_paged_ex(*args, ref))
    del keep
    return out, lse


def attn_decode_paged_noalloc(q, k_pool, v_pool, block_table, seq_lens, max_seq_len: int,
                              softmax_scale: float, *, out, lse=None, status=None, stream=None,
                              dims=None):
    """attn_decode_paged with the library's fixed scratch array instead of a workspace.

    For callers that cannot allocate device memory: out (and lse, if wanted) must be given;
    nothing is allocated here or in the library. Calls that overlap on the GPU race on the
    shared scratch and must be serialized by the caller."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_pool, "k_pool", torch.bfloat16, 4)
    _need(v_pool, "v_pool", torch.bfloat16, 4)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(out, "out", torch.bfloat16, 3)
    B = q.shape[0]
    _rows_at_least("block_table", block_table, B)
    _rows_at_least("seq_lens", seq_lens, B)
    heads = _heads(dims)
    if heads is not None:
        _shape("q", q, (B, heads[0], 128))
        _pools(k_pool, v_pool, heads[1])
        _given(out, "out", torch.bfloat16, (B, heads[0], 128))
        _given(lse, "lse", torch.float32, (B, heads[0]))
    if status is not None:
        _need(status, "status", torch.int32)
    _on_device("attn_decode_paged_noalloc", q, k_pool, v_pool, block_table, seq_lens, out, lse,
               status)
    lib = load()
    _check("attn_decode_paged_noalloc", lib.attn_decode_paged_noalloc(
        _dims(dims), _ptr(q), _ptr(k_pool), _ptr(v_pool), k_pool.shape[0], _ptr(block_table),
        block_table.shape[1], _ptr(seq_lens), q.shape[0], int(max_seq_len), float(softmax_scale),
        _ptr(out), _ptr(lse), _ptr(status), _stream(stream)))
    return out, lse


def attn_prefill_chunk(q, cu_q_lens, k_pool, v_pool, block_table, seq_lens, max_q_len: int,
                       max_seq_len: int, softmax_scale: float, *, out=None, lse=None,
                       workspace=None, status=None, stream=None, want_lse=True, dims=None,
                       max_ctas=None, softcap: float = 0.0, alibi_slopes=None, window: int = 0,
                       prefix_lens=None, max_prefix_len=None, row_start=None):
    """Chunked prefill: q [Tq, Hq, D] packed by cu_q_lens. Returns (out, lse).

    max_ctas: cap on the persistent grid (attn_prefill_chunk_ex); None = the plain call.
    Score options as in attn_decode_paged, row_start per query row [Tq]
    (attn_prefill_chunk_score; a workspace passed in then has prefill_score_workspace_size
    bytes)."""
    call = "attn_prefill_chunk"
    if _FAST is not None:
        o, l = _attn_outputs(q, out, lse, want_lse, stream)
        if _FAST.prefill(q, cu_q_lens, k_pool, v_pool, block_table, seq_lens, max_q_len, max_seq_len,
                         softmax_scale, o, l, workspace, status, _handle(stream), dims, max_ctas, softcap,
                         alibi_slopes, window, prefix_lens, max_prefix_len, row_start):
            return o, l
    dev = _device(call, q, "q", torch.bfloat16)
    pq = _tensor(call, q, "q", torch.bfloat16, dev)
    pcu = _tensor(call, cu_q_lens, "cu_q_lens", torch.int32, dev)
    pk = _tensor(call, k_pool, "k_pool", torch.bfloat16, dev)
    pv = _tensor(call, v_pool, "v_pool", torch.bfloat16, dev)
    pbt = _tensor(call, block_table, "block_table", torch.int32, dev)
    psl = _tensor(call, seq_lens, "seq_lens", torch.int32, dev)
    if not (q.dim() == 3 and k_pool.dim() == v_pool.dim() == 4 and block_table.dim() == 2
            and cu_q_lens.dim() == seq_lens.dim() == 1):
        _need_dims(("q", q, 3), ("cu_q_lens", cu_q_lens, 1), ("k_pool", k_pool, 4),
                   ("v_pool", v_pool, 4), ("block_table", block_table, 2), ("seq_lens", seq_lens, 1))
    B = seq_lens.shape[0]
    Tq, hq, _ = q.shape
    rows, bt_stride = block_table.shape
    _rows_at_least("cu_q_lens", cu_q_lens, B + 1)
    if rows < B:
        _rows_at_least("block_table", block_table, B)
    num_pages = k_pool.shape[0]
    heads = _heads(dims)
    if heads is not None:
        _sized("q", q, (Tq, heads[0], 128))
        pool = (num_pages, 16, heads[1], 128)
        _sized("k_pool", k_pool, pool)
        _sized("v_pool", v_pool, pool)
    if out is None:
        out = _empty(q.shape, torch.bfloat16, q.device, stream)
        po = out.data_ptr()
    else:
        po = _tensor(call, out, "out", torch.bfloat16, dev)
        _sized("out", out, q.shape)
    if lse is None:
        if want_lse:
            lse = _empty((Tq, hq), torch.float32, q.device, stream)
        pl = None if lse is None else lse.data_ptr()
    else:
        pl = _tensor(call, lse, "lse", torch.float32, dev)
        _sized("lse", lse, (Tq, hq))
    max_q_len, max_seq_len = int(max_q_len), int(max_seq_len)
    score = _score(call, dev, hq, B, Tq, max_seq_len, softcap, alibi_slopes, window, prefix_lens,
                   max_prefix_len, row_start)
    if workspace is None:
        nbytes = (_workspace_size(prefill_score_workspace_size, B, Tq, dims) if score is not None
                  else _workspace_size(prefill_workspace_size, B, max_q_len, max_seq_len, dims))
        workspace = _workspace(nbytes, q.device, None, stream)
    else:
        _on_device(call, workspace)
    ps = None if status is None else _tensor(call, status, "status", torch.int32, dev)
    lib = load()
    args = (_dims(dims), pq, pcu, Tq, pk, pv, num_pages, pbt, bt_stride, psl, B, max_q_len,
            max_seq_len, float(softmax_scale), po, pl, workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), ps, _stream(stream))
    keep, ref = _opts(max_ctas)
    if score is not None:
        _check("attn_prefill_chunk_score",
               lib.attn_prefill_chunk_score(*args, ref, ctypes.byref(score)))
    elif ref is None:
        _check(call, lib.attn_prefill_chunk(*args))
    else:
        _check("attn_prefill_chunk_ex", lib.attn_prefill_chunk_ex(*args, ref))
    del keep
    return out, lse


def attn_merge_lse(o_parts, lse_parts, *, out=None, lse_out=None, stream=None):
    """o_parts fp32 [S, R, H, D], lse_parts fp32 [S, R, H] -> (out bf16 [R, H, D], lse [R, H])."""
    _need(o_parts, "o_parts", torch.float32, 4)
    _need(lse_parts, "lse_parts", torch.float32, 3)
    S, R, H, D = o_parts.shape
    _shape("lse_parts", lse_parts, (S, R, H))
    _given(out, "out", torch.bfloat16, (R, H, D))
    _given(lse_out, "lse_out", torch.float32, (R, H))
    if out is None:
        out = torch.empty(R, H, D, dtype=torch.bfloat16, device=o_parts.device)
    if lse_out is None:
        lse_out = torch.empty(R, H, dtype=torch.float32, device=o_parts.device)
    _on_device("attn_merge_lse", o_parts, lse_parts, out, lse_out)
    lib = load()
    _check("attn_merge_lse", lib.attn_merge_lse(S, R, H, D, _ptr(o_parts), _ptr(lse_parts),
                                                _ptr(out), _ptr(lse_out), _stream(stream)))
    return out, lse_out


# ----------------------------------------------------------------------------------------------
# page tables and rotary positions
# ----------------------------------------------------------------------------------------------
StepPlan = collections.namedtuple("StepPlan",
                                  "cu_new_lens seq_lens positions slot_map free_count")


def _new_or_given(call, t, name, dtype, shape, dev, stream):
    """(tensor, data_ptr) of an output: the caller's, checked, or a new one."""
    if t is None:
        t = _empty(shape, dtype, dev, stream)
        return t, t.data_ptr()
    p = _tensor(call, t, name, dtype, dev)
    _sized(name, t, shape)
    return t, p


def paged_step_plan(cached_lens, new_lens, block_table, free_pages, free_count, num_pages: int, *,
                    total_rows: int, free_count_out=None, cu_new_lens=None, seq_lens=None,
                    positions=None, slot_map=None, status=None, stream=None) -> StepPlan:
    """Pages, positions and slots of a step that adds new_lens[b] tokens to request b's
    cached_lens[b]. block_table is updated in place; returns StepPlan(cu_new_lens [B+1],
    seq_lens [B], positions [total_rows], slot_map int64 [total_rows], free_count [1]).

    free_pages[:free_count] are free; pages are taken from its end, in request order. Requests
    that the free pages do not cover are left as they are (their rows get slot -1,
    DEV_ERR_NO_PAGES). free_count_out may be free_count, seq_lens may be cached_lens."""
    call, i32 = "paged_step_plan", torch.int32
    if _FAST is not None and _FAST.step_plan(
            cached_lens, new_lens, block_table, free_pages, free_count, num_pages, total_rows,
            free_count_out, cu_new_lens, seq_lens, positions, slot_map, status, _handle(stream)):
        return StepPlan(cu_new_lens, seq_lens, positions, slot_map, free_count_out)
    dev = _device(call, cached_lens, "cached_lens", i32)
    pc = _tensor(call, cached_lens, "cached_lens", i32, dev)
    pn = _tensor(call, new_lens, "new_lens", i32, dev)
    pbt = _tensor(call, block_table, "block_table", i32, dev)
    pf = _tensor(call, free_pages, "free_pages", i32, dev)
    pfc = _tensor(call, free_count, "free_count", i32, dev)
    if not (cached_lens.dim() == free_pages.dim() == free_count.dim() == 1
            and block_table.dim() == 2):
        _need_dims(("cached_lens", cached_lens, 1), ("block_table", block_table, 2),
                   ("free_pages", free_pages, 1), ("free_count", free_count, 1))
    B = cached_lens.shape[0]
    _sized("new_lens", new_lens, (B,))
    rows, bt_stride = block_table.shape
    if rows < B:
        _rows_at_least("block_table", block_table, B)
    _rows_at_least("free_count", free_count, 1)
    total_rows = int(total_rows)
    if total_rows < 0:
        raise ValueError("total_rows must be >= 0")
    free_count_out, pfo = _new_or_given(call, free_count_out, "free_count_out", i32, (1,), dev,
                                        stream)
    cu_new_lens, pcu = _new_or_given(call, cu_new_lens, "cu_new_lens", i32, (B + 1,), dev, stream)
    seq_lens, psl = _new_or_given(call, seq_lens, "seq_lens", i32, (B,), dev, stream)
    positions, pp = _new_or_given(call, positions, "positions", i32, (total_rows,), dev, stream)
    slot_map, psm = _new_or_given(call, slot_map, "slot_map", torch.int64, (total_rows,), dev,
                                  stream)
    ps = None if status is None else _tensor(call, status, "status", i32, dev)
    _check(call, load().paged_step_plan(
        pc, pn, B, pbt, bt_stride, pf, free_pages.shape[0], pfc, int(num_pages), total_rows, pfo,
        pcu, psl, pp, psm, ps, _stream(stream)))
    return StepPlan(cu_new_lens, seq_lens, positions, slot_map, free_count_out)


def paged_release(begin_pages, end_pages, block_table, free_pages, free_count, num_pages: int, *,
                  free_count_out=None, status=None, stream=None):
    """Append the pages of each request's logical range [begin_pages[b], end_pages[b]) to
    free_pages and set their block_table entries to -1 (entries that are -1 are skipped).
    Returns the new free count [1] (free_count_out, which may be free_count)."""
    call, i32 = "paged_release", torch.int32
    if _FAST is not None and _FAST.release(begin_pages, end_pages, block_table, free_pages, free_count,
                                           num_pages, free_count_out, status, _handle(stream)):
        return free_count_out
    dev = _device(call, begin_pages, "begin_pages", i32)
    pb = _tensor(call, begin_pages, "begin_pages", i32, dev)
    pe = _tensor(call, end_pages, "end_pages", i32, dev)
    pbt = _tensor(call, block_table, "block_table", i32, dev)
    pf = _tensor(call, free_pages, "free_pages", i32, dev)
    pfc = _tensor(call, free_count, "free_count", i32, dev)
    if not (begin_pages.dim() == free_pages.dim() == free_count.dim() == 1
            and block_table.dim() == 2):
        _need_dims(("begin_pages", begin_pages, 1), ("block_table", block_table, 2),
                   ("free_pages", free_pages, 1), ("free_count", free_count, 1))
    B = begin_pages.shape[0]
    _sized("end_pages", end_pages, (B,))
    rows, bt_stride = block_table.shape
    if rows < B:
        _rows_at_least("block_table", block_table, B)
    _rows_at_least("free_count", free_count, 1)
    free_count_out, pfo = _new_or_given(call, free_count_out, "free_count_out", i32, (1,), dev,
                                        stream)
    ps = None if status is None else _tensor(call, status, "status", i32, dev)
    _check(call, load().paged_release(pb, pe, B, pbt, bt_stride, pf, free_pages.shape[0], pfc,
                                      int(num_pages), pfo, ps, _stream(stream)))
    return free_count_out


_ROPE_KINDS = {"none": 0, "linear": 1, "ntk": 2, "llama3": 3, "yarn": 4}


def rope_inv_freq(rot_dim: int = 128, theta: float = 1e6, *, scaling: str = "none",
                  factor: float = 1.0, original_max_position: float = 32768,
                  low_freq_factor: float = 1.0, high_freq_factor: float = 4.0,
                  beta_fast: float = 32.0, beta_slow: float = 1.0, attn_factor: float = 0.0,
                  device=None):
    """Rotary frequencies in 64 bits [rot_dim / 2], stretched for long contexts, and the factor for
    cos and sin: (inv_freq, attn_factor) for rope_append_paged. scaling: none, linear, ntk, llama3
    or yarn (pa_rope_inv_freq). On the current CUDA device unless device says otherwise."""
    if scaling not in _ROPE_KINDS:
        raise ValueError(f"scaling must be one of {sorted(_ROPE_KINDS)}, got {scaling!r}")
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be a positive even number")
    sc = RopeScaling(_ROPE_KINDS[scaling], factor, original_max_position, low_freq_factor,
                     high_freq_factor, beta_fast, beta_slow, attn_factor)
    host = (ctypes.c_double * (rot_dim // 2))()
    a = ctypes.c_float(0.0)
    _check("pa_rope_inv_freq", load().pa_rope_inv_freq(rot_dim, theta, ctypes.byref(sc), host,
                                                       ctypes.byref(a)))
    freq = torch.tensor(list(host), dtype=torch.float64,
                        device="cuda" if device is None else device)
    return freq, float(a.value)


def _rows_strided(call, t, name, dev, T, heads):
    """(data_ptr, row stride) of a [T, heads, 128] bf16 tensor whose rows may lie apart."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.get_device() != dev:
        _on_device(call, t)
    if t.shape != (T, heads, 128):
        raise ValueError(f"{name} must have shape {(T, heads, 128)}, got {tuple(t.shape)}")
    row, head, dim = t.stride()
    if dim != 1 or (head != 128 and heads > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return t.data_ptr(), row if T > 1 else heads * 128


def rope_append_paged(q, k_new, v_new, positions, slot_map, k_pool, v_pool, inv_freq, *,
                      interleaved: bool = False, attn_factor: float = 1.0, q_gamma=None,
                      k_gamma=None, eps: float = 1e-6, q_out=None, status=None, stream=None,
                      dims=None):
    """Rotate (and, with gammas, RMS-normalise per head) q [T, Hq, 128] and k_new [T, Hkv, 128] at
    their positions, write k and v into the pools at slot_map (negative: padding row, left
    alone). Returns q_out [T, Hq, 128]. rot_dim is 2 * len(inv_freq); rows of q, k_new and v_new
    may be strided (slices of one projection)."""
    call = "rope_append_paged"
    if _FAST is not None:
        o, _ = _attn_outputs(q, q_out, None, False, stream)
        if _FAST.rope(q, k_new, v_new, positions, slot_map, k_pool, v_pool, inv_freq,
                      1 if interleaved else 0, attn_factor, q_gamma, k_gamma, eps, o, status,
                      _handle(stream), dims):
            return o
    dev = _device(call, q, "q", torch.bfloat16)
    hq, hkv = _heads(dims) or tuple(dims[:2])  # (other shapes: the library rejects them)
    T = q.shape[0] if q.dim() else 0
    pq, qs = _rows_strided(call, q, "q", dev, T, hq)
    pk, ks = _rows_strided(call, k_new, "k_new", dev, T, hkv)
    pv, vs = _rows_strided(call, v_new, "v_new", dev, T, hkv)
    pp = _tensor(call, positions, "positions", torch.int32, dev)
    psm = _tensor(call, slot_map, "slot_map", torch.int64, dev)
    pif = _tensor(call, inv_freq, "inv_freq", torch.float64, dev)
    _sized("positions", positions, (T,))
    _sized("slot_map", slot_map, (T,))
    if inv_freq.dim() != 1:
        raise ValueError(f"inv_freq must have 1 dim, got {inv_freq.dim()}")
    pkp = _tensor(call, k_pool, "k_pool", torch.bfloat16, dev)
    pvp = _tensor(call, v_pool, "v_pool", torch.bfloat16, dev)
    if k_pool.dim() != 4:
        raise ValueError(f"k_pool must have 4 dims, got {k_pool.dim()}")
    num_pages = k_pool.shape[0]
    _sized("k_pool", k_pool, (num_pages, 16, hkv, 128))
    _sized("v_pool", v_pool, (num_pages, 16, hkv, 128))
    pqg = pkg = None
    if q_gamma is not None:
        pqg = _tensor(call, q_gamma, "q_gamma", torch.float32, dev)
        _sized("q_gamma", q_gamma, (128,))
    if k_gamma is not None:
        pkg = _tensor(call, k_gamma, "k_gamma", torch.float32, dev)
        _sized("k_gamma", k_gamma, (128,))
    q_out, pqo = _new_or_given(call, q_out, "q_out", torch.bfloat16, (T, hq, 128), dev, stream)
    ps = None if status is None else _tensor(call, status, "status", torch.int32, dev)
    _check(call, load().rope_append_paged(
        _dims(dims), 2 * inv_freq.shape[0], 1 if interleaved else 0, pif, float(attn_factor), pq, qs,
        pk, ks, pv, vs, T, pp, psm, pqg, pkg, float(eps), pqo, pkp, pvp, num_pages, ps,
        _stream(stream)))
    return q_out


# ----------------------------------------------------------------------------------------------
# beam search over the paged cache
# ----------------------------------------------------------------------------------------------
def decode_shared_workspace_size(batch: int, groups: int, max_group_rows: int, dims=None) -> int:
    """Workspace of attn_decode_paged_shared."""
    return int(load().pa_decode_shared_workspace_size(_dims(dims), batch, groups, max_group_rows))


def attn_decode_paged_shared(q, k_pool, v_pool, block_table, seq_lens, cu_group_rows, shared_pages,
                             max_seq_len: int, softmax_scale: float, *, max_group_rows=None, out=None,
                             lse=None, workspace=None, status=None, stream=None, want_lse=True,
                             dims=None):
    """attn_decode_paged for rows in groups that share leading pages: rows cu_group_rows[g] ..
    cu_group_rows[g + 1] - 1 have their first shared_pages[g] block-table entries in common, and the
    keys of those pages are read once for the group. q [B, Hq, D]; returns (out, lse).

    max_group_rows: host bound of a group's rows (default: B). Rows in no group share nothing; a row
    with fewer keys than the shared pages hold reads its own entries alone. Weights of pages that more
    than 8 rows share are rounded to bf16, all others are kept as attn_decode_paged keeps them. That call takes
    the same tables and is the quicker one for one group of R rows over n keys while (R - 1) n is below
    about 27,000. No score options and no max_ctas here."""
    call, i32 = "attn_decode_paged_shared", torch.int32
    if _FAST is not None:
        o, l = _attn_outputs(q, out, lse, want_lse, stream)
        if _FAST.decode_shared(q, k_pool, v_pool, block_table, seq_lens, cu_group_rows, shared_pages, max_seq_len,
                               softmax_scale, max_group_rows, o, l, workspace, status, _handle(stream), dims):
            return o, l
    dev = _device(call, q, "q", torch.bfloat16)
    pq = _tensor(call, q, "q", torch.bfloat16, dev)
    pk = _tensor(call, k_pool, "k_pool", torch.bfloat16, dev)
    pv = _tensor(call, v_pool, "v_pool", torch.bfloat16, dev)
    pbt = _tensor(call, block_table, "block_table", i32, dev)
    psl = _tensor(call, seq_lens, "seq_lens", i32, dev)
    pcu = _tensor(call, cu_group_rows, "cu_group_rows", i32, dev)
    psh = _tensor(call, shared_pages, "shared_pages", i32, dev)
    _need_dims(("q", q, 3), ("k_pool", k_pool, 4), ("v_pool", v_pool, 4), ("block_table", block_table, 2),
               ("seq_lens", seq_lens, 1), ("cu_group_rows", cu_group_rows, 1),
               ("shared_pages", shared_pages, 1))
    B, hq, _ = q.shape
    G = shared_pages.shape[0]
    _rows_at_least("block_table", block_table, B)
    _rows_at_least("seq_lens", seq_lens, B)
    if G:
        _rows_at_least("cu_group_rows", cu_group_rows, G + 1)
    num_pages = k_pool.shape[0]
    heads = _heads(dims)
    if heads is not None:
        _sized("q", q, (B, heads[0], 128))
        _sized("k_pool", k_pool, (num_pages, 16, heads[1], 128))
        _sized("v_pool", v_pool, (num_pages, 16, heads[1], 128))
    max_group_rows = B if max_group_rows is None else int(max_group_rows)
    out, po = _new_or_given(call, out, "out", torch.bfloat16, q.shape, dev, stream)
    pl = None
    if lse is not None or want_lse:
        lse, pl = _new_or_given(call, lse, "lse", torch.float32, (B, hq), dev, stream)
    if workspace is None:
        nbytes = _workspace_size(decode_shared_workspace_size, B, G, max_group_rows, dims)
        workspace = _workspace(nbytes, q.device, None, stream)
    else:
        _on_device(call, workspace)
    ps = None if status is None else _tensor(call, status, "status", i32, dev)
    _check(call, load().attn_decode_paged_shared(
        _dims(dims), pq, pk, pv, num_pages, pbt, block_table.shape[1], psl, B, pcu, psh, G, max_group_rows,
        int(max_seq_len), float(softmax_scale), po, pl, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), ps, _stream(stream)))
    return out, lse


BeamStep = collections.namedtuple("BeamStep", "scores parents tokens live")
_LOGITS = {torch.bfloat16: 0, torch.float32: 1}


def beam_workspace_size(requests: int, beams: int, vocab: int, k: int) -> int:
    """Workspace of beam_select."""
    return int(load().pa_beam_workspace_size(requests, beams, vocab, k))


def beam_select(logits, scores, k: int, *, live=None, eos_token: int = -1, out_scores=None, parents=None,
                tokens=None, live_out=None, workspace=None, stream=None) -> BeamStep:
    """The k best of each request's candidates scores[n, b] + log_softmax(logits[n, b])[v]: BeamStep(scores
    fp32, parents (b), tokens (v), live int32), each [N, k], best first, equal scores in the order of
    (b, v).

    logits [N, W, V] bf16 or fp32 (rows may lie apart); scores fp32 [N, W], -inf for a beam that is not
    in use; live int32 [N, W]: 0 for a beam that has ended (its one candidate is itself, with eos_token).
    live of the result is 0 for beams that have ended, now or before: the new_lens of paged_step_plan.
    Places without a candidate are (-inf, -1, -1, 0). out_scores may be scores and live_out may be live
    where k is W."""
    call, i32 = "beam_select", torch.int32
    if _FAST is not None:
        made = _FAST.beam(logits, scores, k, live, eos_token, out_scores, parents, tokens, live_out, workspace,
                          _handle(stream))
        if made:
            return BeamStep._make(made)
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a tensor")
    if logits.dtype not in _LOGITS:
        raise TypeError(f"logits must be {torch.bfloat16} or {torch.float32}, got {logits.dtype}")
    dev = _device(call, logits, "logits", logits.dtype)
    if logits.dim() != 3:
        raise ValueError(f"logits must have 3 dims, got {logits.dim()}")
    N, W, V = logits.shape
    s0, s1, s2 = logits.stride()
    if N and W > 1:
        stride = s1
    elif N > 1:
        stride = s0
    else:
        stride = V
    if N and ((V > 1 and s2 != 1) or (N > 1 and W > 1 and s0 != W * s1) or stride < V):
        raise ValueError("logits: a row must be contiguous, and rows equally far apart")
    psc = _tensor(call, scores, "scores", torch.float32, dev)
    _sized("scores", scores, (N, W))
    plv = None
    if live is not None:
        plv = _tensor(call, live, "live", i32, dev)
        _sized("live", live, (N, W))
    k = int(k)
    shape = (N, max(k, 0))
    out_scores, po = _new_or_given(call, out_scores, "out_scores", torch.float32, shape, dev, stream)
    parents, pp = _new_or_given(call, parents, "parents", i32, shape, dev, stream)
    tokens, pt = _new_or_given(call, tokens, "tokens", i32, shape, dev, stream)
    live_out, pl = _new_or_given(call, live_out, "live_out", i32, shape, dev, stream)
    if workspace is None:
        nbytes = _workspace_size(beam_workspace_size, N, W, V, k)
        workspace = _workspace(nbytes, logits.device, None, stream)
    else:
        _on_device(call, workspace)
    _check(call, load().beam_select(
        logits.data_ptr(), _LOGITS[logits.dtype], stride, N, W, V, psc, plv, k, int(eos_token), po, pp, pt,
        pl, workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream)))
    return BeamStep(out_scores, parents, tokens, live_out)


ForkPlan = collections.namedtuple("ForkPlan", "seq_lens copies shared_pages free_count")


def fork_workspace_size(groups: int, beams: int, bt_stride: int) -> int:
    """Workspace of paged_fork."""
    return int(load().pa_fork_workspace_size(groups, beams, bt_stride))


def paged_fork(parents, seq_lens, block_table, free_pages, free_count, num_pages: int, *,
               free_count_out=None, seq_lens_out=None, copies=None, shared_pages=None, workspace=None,
               status=None, stream=None) -> ForkPlan:
    """Row g * W + b of block_table continues row g * W + parents[g, b] (parents int32 [G, W]; -1: the row
    becomes empty): it gets that row's pages, shared between the rows of a group. block_table and
    free_pages are updated in place; returns ForkPlan(seq_lens [G * W], copies [G * W, 3] for
    paged_copy_pages, shared_pages [G] for attn_decode_paged_shared, free_count [1]).

    A child that shares a partly filled last page with an earlier child gets a page of its own from the
    free list, and its copy in copies; pages that no row of the group holds any more go to the list. If
    the free pages do not cover the copies nothing changes (DEV_ERR_NO_PAGES). seq_lens_out may be
    seq_lens, free_count_out may be free_count."""
    call, i32 = "paged_fork", torch.int32
    if _FAST is not None:
        made = _FAST.fork(parents, seq_lens, block_table, free_pages, free_count, num_pages, seq_lens_out, copies,
                          shared_pages, free_count_out, workspace, status, _handle(stream))
        if made:
            return ForkPlan._make(made)
    dev = _device(call, parents, "parents", i32)
    ppa = _tensor(call, parents, "parents", i32, dev)
    psl = _tensor(call, seq_lens, "seq_lens", i32, dev)
    pbt = _tensor(call, block_table, "block_table", i32, dev)
    pf = _tensor(call, free_pages, "free_pages", i32, dev)
    pfc = _tensor(call, free_count, "free_count", i32, dev)
    _need_dims(("parents", parents, 2), ("seq_lens", seq_lens, 1), ("block_table", block_table, 2),
               ("free_pages", free_pages, 1), ("free_count", free_count, 1))
    G, W = parents.shape
    B, stride = G * W, block_table.shape[1]
    _sized("seq_lens", seq_lens, (B,))
    _rows_at_least("block_table", block_table, B)
    _rows_at_least("free_count", free_count, 1)
    free_count_out, pfo = _new_or_given(call, free_count_out, "free_count_out", i32, (1,), dev, stream)
    seq_lens_out, pso = _new_or_given(call, seq_lens_out, "seq_lens_out", i32, (B,), dev, stream)
    copies, pc = _new_or_given(call, copies, "copies", i32, (B, 3), dev, stream)
    shared_pages, psh = _new_or_given(call, shared_pages, "shared_pages", i32, (G,), dev, stream)
    if workspace is None:
        workspace = _workspace(_workspace_size(fork_workspace_size, G, W, stride), parents.device, None, stream)
    else:
        _on_device(call, workspace)
    ps = None if status is None else _tensor(call, status, "status", i32, dev)
    _check(call, load().paged_fork(
        ppa, psl, G, W, pbt, stride, pf, free_pages.shape[0], pfc, int(num_pages), pfo, pso, pc, psh,
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), ps, _stream(stream)))
    return ForkPlan(seq_lens_out, copies, shared_pages, free_count_out)


def paged_copy_pages(copies, pools, *, status=None, stream=None, dims=None):
    """Copy the first copies[i, 2] tokens of page copies[i, 0] to page copies[i, 1] in every pool of
    `pools` (the K and V pools of all layers, bf16 [num_pages, 16, Hkv, 128] of one shape). copies int32
    [rows, 3]; rows of (-1, -1, 0) copy nothing."""
    call = "paged_copy_pages"
    if _FAST is not None and _FAST.copy_pages(copies, pools, status, _handle(stream), dims):
        return
    dev = _device(call, copies, "copies", torch.int32)
    pc = _tensor(call, copies, "copies", torch.int32, dev)
    _shape("copies", copies, (None, 3))
    heads = _heads(dims)
    ptrs = (ctypes.c_void_p * max(1, len(pools)))()
    shape = pools[0].shape if len(pools) and isinstance(pools[0], torch.Tensor) else None
    if heads is not None and shape is not None:
        _shape("pools[0]", pools[0], (None, 16, heads[1], 128))
    for i, t in enumerate(pools):
        ptrs[i] = _tensor(call, t, f"pools[{i}]", torch.bfloat16, dev)
        _sized(f"pools[{i}]", t, shape)
    ps = None if status is None else _tensor(call, status, "status", torch.int32, dev)
    _check(call, load().paged_copy_pages(
        _dims(dims), pc, copies.shape[0], ptrs, len(pools), shape[0] if shape is not None else 1, ps,
        _stream(stream)))


def adaptor_workspace_size(num_frames: int) -> int:
    return int(load().pa_adaptor_workspace_size(num_frames))


def adaptor_mlp_merge4(frames, w1, b1, w2, b2, gamma, beta, eps: float = 1e-5, *, out=None,
                       workspace=None, status=None, stream=None):
    """Decoder embeddings from encoder frames [T_enc, 1024]: 4x merge, Linear-SiLU-Linear-
    LayerNorm. Returns out bf16 [T_enc / 4, 1024]."""
    _need(frames, "frames", torch.bfloat16, 2)
    _need(w1, "w1", torch.bfloat16, 2)
    _need(w2, "w2", torch.bfloat16, 2)
    for t, n in ((b1, "b1"), (b2, "b2"), (gamma, "gamma"), (beta, "beta")):
        _need(t, n, torch.float32, 1)
    n_frames = frames.shape[0]
    T = n_frames // 4
    _shape("frames", frames, (n_frames, 1024))
    _shape("w1", w1, (1024, 4096))
    _shape("w2", w2, (1024, 1024))
    for t, n in ((b1, "b1"), (b2, "b2"), (gamma, "gamma"), (beta, "beta")):
        _shape(n, t, (1024,))
    _given(out, "out", torch.bfloat16, (T, 1024))
    if out is None:
        out = torch.empty(T, 1024, dtype=torch.bfloat16, device=frames.device)
    if workspace is None:
        workspace = torch.empty(max(256, adaptor_workspace_size(n_frames)), dtype=torch.uint8,
                                device=frames.device)
    if status is not None:
        _need(status, "status", torch.int32)
    _on_device("adaptor_mlp_merge4", frames, w1, b1, w2, b2, gamma, beta, out, workspace, status)
    lib = load()
    _check("adaptor_mlp_merge4", lib.adaptor_mlp_merge4(
        n_frames, _ptr(frames), _ptr(w1), _ptr(b1), _ptr(w2), _ptr(b2), _ptr(gamma), _ptr(beta),
        float(eps), _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(status), _stream(stream)))
    return out


def debug_decode_starve(enable: bool) -> None:
    """Test hook: later decode launches of this thread leave one ring stage empty and bound
    their waits by 1 ms, so the bounded-wait give-up path runs (status PA_DEV_ERR_TIMEOUT)."""
    _check("pa_debug_decode_starve", load().pa_debug_decode_starve(1 if enable else 0))


def read_device_status(status, stream=None) -> int:
    """Wait for the stream, return the device status bits and clear them."""
    _need(status, "status", torch.int32)
    flags = ctypes.c_uint32(0)
    _check("pa_read_device_status", load().pa_read_device_status(_ptr(status), ctypes.byref(flags),
                                                                 _stream(stream)))
    return int(flags.value)
