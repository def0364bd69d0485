"""paged_kv_decode_np_gb300 -- GB300 (sm_103a) batched paged-attention decode.

A thin ctypes binding over ``libnp_paged.so`` (C ABI in
``include/np_paged.h``).  The functions keep the C names and only marshal
arguments: every step of the append, the read and the reduce runs in the
library's CUDA kernels.  torch supplies device memory and streams.  There is
no CPU fallback: if the library is missing, or a tensor is not on a CUDA
device, the call raises.

Typical decode step::

    import paged_kv_decode_np_gb300 as npg
    S = npg.np_paged_decode_plan(rows, q_heads, kv_heads, head_dim, block_size,
                                 max_blocks_per_row, torch.bfloat16)
    ws = npg.workspace(rows, q_heads, head_dim, S, device="cuda")   # zeroed
    npg.np_paged_append_decode(out if S <= 1 else None, q, k_new, v_new,
                               slot_mapping, k_pool, v_pool, block_tables,
                               context_lens, scale, num_splits=S, workspace=ws)
    if S > 1:
        npg.np_paged_decode_reduce(out, ws, num_splits=S)

S == 0 (the balanced read) writes ``out`` itself; S > 1 leaves split
partials for np_paged_decode_reduce.  A loop that runs the same step on the
same buffers again and again can check and convert the arguments once::

    step = npg.PreparedStep(out, q, k_new, v_new, slot_mapping, k_pool, v_pool,
                            block_tables, context_lens, scale, S, ws)
    step.launch()   # the same library calls, ~4 us of host time

A prompt, or a chunk of one, of several rows (rotated, appended, attended)::

    table = npg.rope_table(max_positions, head_dim)
    ws = npg.prefill_workspace(head_dim)
    npg.prefill_step(out, q, k_new, v_new, slot_mapping, k_pool, v_pool,
                     block_tables, context_lens, query_starts, scale, ws,
                     cos_sin=table, positions=positions)

The new tokens of a decode step are rotated and appended by np_rope_append,
then read by np_paged_decode.

A cache in 8 bits (q8_pools) is filled by np_kv_append_q8 and read by
np_paged_decode_q8 and np_paged_prefill_q8 (decode_step_q8, prefill_step_q8);
np_block_map keeps a batch's block tables, lengths and slots on the GPU.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

import torch

__all__ = [
    "load", "NPError", "np_abi_version", "np_status_string", "np_kv_append",
    "np_paged_decode_plan", "np_paged_decode_split_len",
    "np_paged_decode_workspace_bytes", "np_paged_decode", "np_paged_decode_reduce",
    "np_paged_decode_noalloc", "NP_NOALLOC_SCRATCH_BYTES", "np_paged_append_decode",
    "np_selftest_bounded_wait", "np_rope_append", "np_paged_prefill",
    "np_paged_prefill_workspace_bytes", "rope_table", "prefill_workspace", "prefill_step",
    "NP_PREFILL_WORKSPACE_BYTES", "workspace", "decode_step", "PreparedStep", "NP_OK", "NP_ERR_INVALID_ARG",
    "NP_ERR_UNSUPPORTED",
    "NP_ERR_WORKSPACE", "NP_ERR_OUT_OF_RANGE", "NP_ERR_CUDA", "NP_F32", "NP_BF16",
    "NP_FLAG_BLOCK_ID", "NP_FLAG_CONTEXT", "NP_FLAG_SLOT", "NP_FLAG_TIMEOUT", "NP_FLAG_CONFIG",
    "NP_FLAG_POSITION", "NP_FLAG_QUERY", "NP_FLAG_VALUE", "NP_FLAG_BLOCKS", "NP_E4M3", "NP_INT8",
    "np_block_map", "np_kv_append_q8", "np_paged_decode_q8", "np_paged_decode_q8_workspace_bytes",
    "np_paged_prefill_q8", "q8_pools", "decode_q8_workspace", "decode_step_q8", "prefill_step_q8",
    "NP_DECODE_Q8_WORKSPACE_BYTES",
]

NP_OK = 0
NP_ERR_INVALID_ARG = 1
NP_ERR_UNSUPPORTED = 2
NP_ERR_WORKSPACE = 3
NP_ERR_OUT_OF_RANGE = 4
NP_ERR_CUDA = 5

NP_F32 = 0
NP_BF16 = 1

NP_FLAG_BLOCK_ID = 0x1
NP_FLAG_CONTEXT = 0x2
NP_FLAG_SLOT = 0x4
NP_FLAG_TIMEOUT = 0x8
NP_FLAG_CONFIG = 0x10
NP_FLAG_POSITION = 0x20
NP_FLAG_QUERY = 0x40
NP_FLAG_VALUE = 0x80
NP_FLAG_BLOCKS = 0x100

NP_E4M3 = 0
NP_INT8 = 1

NP_NOALLOC_SCRATCH_BYTES = 32 << 20
NP_PREFILL_WORKSPACE_BYTES = 64 << 20
NP_DECODE_Q8_WORKSPACE_BYTES = 64 << 20

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libnp_paged.so")

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_LIB: ctypes.CDLL | None = None


class NPError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        name = load().np_status_string(status).decode() if _LIB else str(status)
        super().__init__(f"{call} returned {name}")


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libnp_paged.so (built by ``__graft_entry__.build()``)."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is not built; run `python -c 'import __graft_entry__ as g; "
                           "g.build()'` (nvcc, sm_103a)")
    lib = ctypes.CDLL(p)
    lib.np_status_string.restype = ctypes.c_char_p
    lib.np_status_string.argtypes = [ctypes.c_int]
    lib.np_abi_version.restype = _I32
    lib.np_abi_version.argtypes = []
    lib.np_kv_append.restype = ctypes.c_int
    lib.np_kv_append.argtypes = [_P, _P, ctypes.c_int, _I64, _I32, _I32, _I32, _P, _P, _P,
                                 _I32, _P, _P]
    lib.np_paged_decode_plan.restype = ctypes.c_int
    lib.np_paged_decode_plan.argtypes = [_I32, _I32, _I32, _I32, _I32, _I32, ctypes.c_int,
                                         _I32, ctypes.POINTER(_I32)]
    lib.np_paged_decode_split_len.restype = _I64
    lib.np_paged_decode_split_len.argtypes = [_I32, _I32, _I32]
    lib.np_paged_decode_workspace_bytes.restype = ctypes.c_size_t
    lib.np_paged_decode_workspace_bytes.argtypes = [_I32, _I32, _I32, _I32]
    lib.np_paged_decode.restype = ctypes.c_int
    lib.np_paged_decode.argtypes = [_P, _P, _P, _P, ctypes.c_int, _I64, _I32, _I32, _I32, _P,
                                    _I32, _P, _I32, _I32, _I32, ctypes.c_float, _I32, _P,
                                    ctypes.c_size_t, _P, _P]
    lib.np_paged_append_decode.restype = ctypes.c_int
    lib.np_paged_append_decode.argtypes = [_P, _P, _P, _P, _P, _P, _P, ctypes.c_int, _I64, _I32,
                                           _I32, _I32, _P, _I32, _P, _I32, _I32, _I32,
                                           ctypes.c_float, _I32, _P, ctypes.c_size_t, _P, _P]
    lib.np_paged_decode_noalloc.restype = ctypes.c_int
    lib.np_paged_decode_noalloc.argtypes = [_P, _P, _P, _P, ctypes.c_int, _I64, _I32, _I32, _I32,
                                            _P, _I32, _P, _I32, _I32, _I32, ctypes.c_float, _I32,
                                            _P, _P]
    lib.np_paged_decode_reduce.restype = ctypes.c_int
    lib.np_paged_decode_reduce.argtypes = [_P, ctypes.c_int, _P, ctypes.c_size_t, _I32, _I32,
                                           _I32, _I32, _P]
    lib.np_selftest_bounded_wait.restype = ctypes.c_int
    lib.np_selftest_bounded_wait.argtypes = [_P, _I64, _P]
    if hasattr(lib, "np_rope_append"):  # a library of ABI version 2 has no prompt side
        _declare_prompt(lib)
    if hasattr(lib, "np_block_map"):  # a library of ABI version 3 has no 8-bit cache
        _declare_q8(lib)
    if path is None:
        _LIB = lib
    return lib


def _declare_prompt(lib: ctypes.CDLL) -> None:
    lib.np_rope_append.restype = ctypes.c_int
    lib.np_rope_append.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P, ctypes.c_int, _I64,
                                   _I32, _I32, _I32, _I32, _P, _I32, _I32, _P, _I32,
                                   ctypes.POINTER(_I32), _I32, _P, _P, ctypes.c_float, _I32, _P,
                                   _P]
    for name in ("np_rope_append_packed", "np_paged_prefill_packed", "np_paged_prefill_check"):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = [ctypes.c_char_p]
    lib.np_paged_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.np_paged_prefill_workspace_bytes.argtypes = [_I32]
    lib.np_paged_prefill.restype = ctypes.c_int
    lib.np_paged_prefill.argtypes = [_P, _P, _P, _P, ctypes.c_int, _I64, _I32, _I32, _I32, _P, _I32,
                                     _P, _P, _I32, _I32, _I32, ctypes.c_float, _P, ctypes.c_size_t,
                                     _P, _P]


def _declare_q8(lib: ctypes.CDLL) -> None:
    for name in ("np_block_map_packed", "np_kv_append_q8_packed", "np_paged_decode_q8_packed",
                 "np_paged_decode_q8_check", "np_paged_prefill_q8_packed", "np_paged_prefill_q8_check"):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = [ctypes.c_char_p]
    lib.np_paged_decode_q8_workspace_bytes.restype = ctypes.c_size_t
    lib.np_paged_decode_q8_workspace_bytes.argtypes = [_I32]


def _check(status: int, call: str) -> None:
    if status != NP_OK:
        raise NPError(status, call)


def _dtype_code(dt) -> int:
    if dt in (torch.float32, "f32", NP_F32):
        return NP_F32
    if dt in (torch.bfloat16, "bf16", NP_BF16):
        return NP_BF16
    raise TypeError(f"unsupported dtype {dt}; the library stores float32 or bfloat16")


def _current_device() -> int:
    """The CUDA device the library's kernels launch on: torch's current one
    (the stream, the tensor maps and the no-allocation scratch all belong
    to it); -1 where CUDA cannot initialise, so that the tensors' own check
    reports the problem."""
    try:
        return torch.cuda.current_device()
    except (RuntimeError, AssertionError):
        return -1


def _dev(t: torch.Tensor, name: str, cur: int) -> int:
    """The device address of ``t``, after checking that it is a contiguous
    tensor on device ``cur`` (a tensor on another GPU would be dereferenced
    by kernels running on this one)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (no CPU path exists)")
    if t.device.index != cur:
        raise ValueError(f"{name} is on {t.device} but the current device is cuda:{cur}; "
                         "call inside torch.cuda.device(...) of the tensors' GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _opt(t: torch.Tensor | None, name: str, cur: int) -> int | None:
    return None if t is None else _dev(t, name, cur)


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        if stream.device.index != _current_device():
            raise ValueError(f"stream is on {stream.device} but the current device is "
                             f"cuda:{_current_device()}")
        return stream.cuda_stream
    return int(stream)


def _q_shape(q: torch.Tensor, name: str = "q"):
    """(rows, query_len, q_heads, head_dim) of a [R, Hq, D] or [R, Q, Hq, D] tensor."""
    if q.dim() == 3:
        return q.shape[0], 1, q.shape[1], q.shape[2]
    if q.dim() == 4:
        return tuple(q.shape)
    raise ValueError(f"{name} must be [rows, q_heads, head_dim] or "
                     "[rows, query_len, q_heads, head_dim]")


def np_abi_version() -> int:
    return load().np_abi_version()


def np_status_string(status: int) -> str:
    return load().np_status_string(status).decode()


def np_kv_append(k_pool, v_pool, k_new, v_new, slot_mapping, err_word=None, stream=None):
    """Scatter [T, Hk, D] new K/V rows into the pools at ``slot_mapping`` (int64 [T]).

    Leading dimensions are flattened: [R, Q, Hk, D] tokens with [R, Q] slots
    are R*Q tokens.
    """
    nb, bs, hk, d = k_pool.shape
    if k_new.dim() > 3:
        k_new, v_new = k_new.reshape(-1, hk, d), v_new.reshape(-1, hk, d)
        slot_mapping = slot_mapping.reshape(-1)
    if v_pool.shape != k_pool.shape or k_new.shape != v_new.shape or \
            k_new.shape[1:] != (hk, d) or k_new.dtype != k_pool.dtype or \
            v_new.dtype != k_pool.dtype or v_pool.dtype != k_pool.dtype:
        raise ValueError("np_kv_append: shape/dtype mismatch")
    if slot_mapping.dtype != torch.int64 or slot_mapping.shape != (k_new.shape[0],):
        raise ValueError("np_kv_append: slot_mapping must be int64 [num_tokens]")
    cur = _current_device()
    st = load().np_kv_append(
        _dev(k_pool, "k_pool", cur), _dev(v_pool, "v_pool", cur), _dtype_code(k_pool.dtype), nb,
        bs, hk, d, _dev(k_new, "k_new", cur), _dev(v_new, "v_new", cur),
        _dev(slot_mapping, "slot_mapping", cur), k_new.shape[0], _opt(err_word, "err_word", cur),
        _stream(stream))
    _check(st, "np_kv_append")


def rope_table(max_positions: int, rot_dim: int, base: float = 10000.0, inv_freq=None,
               device="cuda") -> torch.Tensor:
    """np_rope_append's table: fp32 [max_positions, rot_dim], row p the cosines
    of the rot_dim/2 pairs' angles p * inv_freq[j] and then their sines, formed
    in 64 bits (a far position's angle has lost its fraction in 32).
    ``inv_freq`` (rot_dim/2 values) replaces base ** (-2 j / rot_dim)."""
    half = rot_dim // 2
    if inv_freq is None:
        f = float(base) ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    else:
        f = torch.as_tensor(inv_freq, device=device).to(torch.float64)
        if f.shape != (half,):
            raise ValueError("rope_table: inv_freq must have rot_dim/2 values")
    ang = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


# np_rope_append_args and np_paged_prefill_args (np_paged.h): a foreign call
# converts one argument instead of thirty, which is most of a small call's time.
_ROPE_ARGS = struct.Struct("@13P4q15if")
_PREFILL_ARGS = struct.Struct("@10P2q8if")


def _device_now() -> int:
    """torch's current CUDA device (as _current_device, without its lazy
    initialisation: a CUDA tensor exists wherever the answer matters); -2, no
    tensor's device, where there is none."""
    try:
        cur = torch._C._cuda_getDevice()
    except (RuntimeError, AttributeError):
        cur = _current_device()
    return cur if cur >= 0 else -2


class _Codes(dict):
    def __missing__(self, dt):
        return _dtype_code(dt)  # raises


_CODES = _Codes({torch.float32: NP_F32, torch.bfloat16: NP_BF16})


def _refuse(cur: int, **tensors) -> None:
    """_dev's refusal of the first tensor that is not a contiguous one on
    device ``cur`` (the calls below look at all of theirs in one condition)."""
    for name, t in tensors.items():
        if t is not None:
            _dev(t, name, cur)


def _stream_now(stream, cur: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(cur)
    return _stream(stream) or 0


def _pack(form: struct.Struct, call: str, *values) -> bytes:
    try:
        return form.pack(*values)
    except struct.error as e:
        raise ValueError(f"{call}: a size does not fit its type ({e})") from None


def _token_rows(t: torch.Tensor, name: str, cur: int, n: int, heads: int, d: int):
    """(address, elements between tokens) of a [n, heads, d] tensor whose heads
    are dense; its tokens may lie further apart (a view of wider rows)."""
    if t.get_device() != cur:
        _dev(t, name, cur)  # raises
    s0, s1, s2 = t.stride()
    if n > 0 and (s2 != 1 or (heads > 1 and s1 != d)):
        raise ValueError(f"{name}: heads and dims must be dense (only tokens may be strided)")
    return t.data_ptr(), (s0 if n > 1 else heads * d)


def np_rope_append(q_out, q, k_new, v_new, slot_mapping, k_pool, v_pool, cos_sin, positions,
                   sections=None, interleaved: bool = False, q_weight=None, k_weight=None,
                   eps: float = 1e-6, err_word=None, stream=None):
    """Normalise (where a weight is given) and rotate the new tokens' q and k;
    q goes to ``q_out`` (which may be ``q``), k and v to their pool slots (see
    np_paged.h).

    q [T, q_heads, head_dim], k_new/v_new [T, kv_heads, head_dim]: views whose
    tokens are strided (slices of a fused projection's rows) are taken as they
    are.  slot_mapping int64 [T]; cos_sin fp32 [max_positions, rot_dim] (see
    rope_table); positions int32 [T], or [axes, T] with ``sections`` pairs per
    axis.  q and q_out None: k and v only.
    """
    name = "np_rope_append"
    nb, bs, hk, d = k_pool.shape
    dt = k_pool.dtype
    if k_new.dim() != 3 or v_pool.shape != k_pool.shape or k_new.shape != v_new.shape:
        raise ValueError(f"{name}: k_new/v_new must be [tokens, kv_heads, head_dim] of the pools")
    n, h1, d1 = k_new.shape
    if h1 != hk or d1 != d:
        raise ValueError(f"{name}: k_new/v_new must be [tokens, kv_heads, head_dim] of the pools")
    if v_pool.dtype is not dt or k_new.dtype is not dt or v_new.dtype is not dt:
        raise ValueError(f"{name}: k_new, v_new and the pools must share a dtype")
    hq = 0
    if (q is None) != (q_out is None) or (q is None and q_weight is not None):
        raise ValueError(f"{name}: q and q_out go together")
    if q is not None:
        if q.dim() != 3 or q.dtype is not dt:
            raise ValueError(f"{name}: q must be [tokens, q_heads, head_dim] of the pools' dtype")
        n1, hq, d1 = q.shape
        if n1 != n or d1 != d:
            raise ValueError(f"{name}: q must be [tokens, q_heads, head_dim] of the pools' dtype")
        if q_out.shape != q.shape or q_out.dtype is not dt:
            raise ValueError(f"{name}: q_out must match q")
        if hq == 0:
            raise ValueError(f"{name}: q has no heads; pass q and q_out as None")
    if q_weight is not None and (q_weight.dtype is not dt or q_weight.shape != (d,)):
        raise ValueError(f"{name}: q_weight must be [head_dim] of the pools' dtype")
    if k_weight is not None and (k_weight.dtype is not dt or k_weight.shape != (d,)):
        raise ValueError(f"{name}: k_weight must be [head_dim] of the pools' dtype")
    if slot_mapping.dtype is not torch.int64 or slot_mapping.shape != (n,):
        raise ValueError(f"{name}: slot_mapping must be int64 [tokens]")
    if cos_sin.dtype is not torch.float32 or cos_sin.dim() != 2:
        raise ValueError(f"{name}: cos_sin must be float32 [max_positions, rot_dim]")
    dims = positions.dim()
    if positions.dtype is not torch.int32 or dims not in (1, 2) or positions.shape[-1] != n:
        raise ValueError(f"{name}: positions must be int32 [tokens] or [axes, tokens]")
    axes = 1 if dims == 1 else positions.shape[0]
    sec = (0, 0, 0, 0)
    if sections is not None:
        if len(sections) != axes:
            raise ValueError(f"{name}: one section per position axis")
        sec = (tuple(sections) + sec)[:4]  # more than four axes: refused by the library
    cur = _device_now()
    qp, qs = (0, 0) if q is None else _token_rows(q, "q", cur, n, hq, d)
    kp, ks = _token_rows(k_new, "k_new", cur, n, hk, d)
    vp, vs = _token_rows(v_new, "v_new", cur, n, hk, d)
    max_pos, rot = cos_sin.shape
    if not (slot_mapping.get_device() == k_pool.get_device() == v_pool.get_device() ==
            cos_sin.get_device() == positions.get_device() == cur and
            (q_out is None or (q_out.get_device() == cur and q_out.is_contiguous())) and
            (q_weight is None or (q_weight.get_device() == cur and q_weight.is_contiguous())) and
            (k_weight is None or (k_weight.get_device() == cur and k_weight.is_contiguous())) and
            (err_word is None or (err_word.get_device() == cur and err_word.is_contiguous())) and
            slot_mapping.is_contiguous() and k_pool.is_contiguous() and v_pool.is_contiguous() and
            cos_sin.is_contiguous() and positions.is_contiguous()):
        _refuse(cur, q_out=q_out, slot_mapping=slot_mapping, k_pool=k_pool, v_pool=v_pool,
                cos_sin=cos_sin, positions=positions, q_weight=q_weight, k_weight=k_weight,
                err_word=err_word)
    st = load().np_rope_append_packed(_pack(
        _ROPE_ARGS, name, 0 if q_out is None else q_out.data_ptr(), qp, kp, vp,
        slot_mapping.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), cos_sin.data_ptr(),
        positions.data_ptr(), 0 if q_weight is None else q_weight.data_ptr(),
        0 if k_weight is None else k_weight.data_ptr(),
        0 if err_word is None else err_word.data_ptr(), _stream_now(stream, cur),
        qs, ks, vs, nb, _CODES[dt], bs, hq, hk, d, max_pos, rot, axes,
        1 if interleaved else 0, n, 0 if sections is None else 1, *sec, eps))
    if st != NP_OK:
        raise NPError(st, name)


def np_paged_prefill_workspace_bytes(head_dim) -> int:
    return load().np_paged_prefill_workspace_bytes(head_dim)


def prefill_workspace(head_dim, device="cuda") -> torch.Tensor:
    """A workspace for np_paged_prefill (its contents need no initialisation)."""
    n = np_paged_prefill_workspace_bytes(head_dim)
    if n == 0:
        raise ValueError(f"unsupported head_dim {head_dim}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def np_paged_prefill(out, q, k_pool, v_pool, block_tables, context_lens, query_starts, scale,
                     workspace, err_word=None, stream=None):
    """Attention of ragged chunks of new tokens over the paged cache (see
    np_paged.h).  q/out [tokens, q_heads, head_dim]; query_starts int32
    [rows + 1]; row r's chunk q[query_starts[r]:query_starts[r + 1]] holds its
    newest positions, already appended to the pools."""
    _launch_prefill(_prefill_args(out, q, k_pool, v_pool, block_tables, context_lens, query_starts,
                                  scale, workspace, err_word, stream))


def _launch_prefill(packed: bytes) -> None:
    st = load().np_paged_prefill_packed(packed)
    if st != NP_OK:
        raise NPError(st, "np_paged_prefill")


def _prefill_args(out, q, k_pool, v_pool, block_tables, context_lens, query_starts, scale,
                  workspace, err_word, stream) -> bytes:
    """np_paged_prefill's packed arguments, after the binding's checks."""
    name = "np_paged_prefill"
    if q.dim() != 3 or k_pool.dim() != 4:
        raise ValueError(f"{name}: q must be [tokens, q_heads, head_dim]")
    nb, bs, hk, d = k_pool.shape
    tokens, hq, d1 = q.shape
    dt = q.dtype
    if d1 != d or v_pool.shape != k_pool.shape or k_pool.dtype is not dt or v_pool.dtype is not dt:
        raise ValueError(f"{name}: q/pool shape or dtype mismatch")
    if out.shape != q.shape or out.dtype is not dt:
        raise ValueError(f"{name}: out must match q")
    if block_tables.dtype is not torch.int32 or block_tables.dim() != 2:
        raise ValueError(f"{name}: block_tables must be int32 [rows, max_blocks]")
    rows, mb = block_tables.shape
    if context_lens.dtype is not torch.int32 or context_lens.shape != (rows,):
        raise ValueError(f"{name}: context_lens must be int32 [rows]")
    if query_starts.dtype is not torch.int32 or query_starts.shape != (rows + 1,):
        raise ValueError(f"{name}: query_starts must be int32 [rows + 1]")
    cur = _device_now()
    if not (out.get_device() == q.get_device() == k_pool.get_device() == v_pool.get_device() ==
            block_tables.get_device() == context_lens.get_device() ==
            query_starts.get_device() == cur and
            (workspace is None or (workspace.get_device() == cur and workspace.is_contiguous())) and
            (err_word is None or (err_word.get_device() == cur and err_word.is_contiguous())) and
            out.is_contiguous() and q.is_contiguous() and k_pool.is_contiguous() and
            v_pool.is_contiguous() and block_tables.is_contiguous() and
            context_lens.is_contiguous() and query_starts.is_contiguous()):
        _refuse(cur, out=out, q=q, k_pool=k_pool, v_pool=v_pool, block_tables=block_tables,
                context_lens=context_lens, query_starts=query_starts, workspace=workspace,
                err_word=err_word)
    return _pack(
        _PREFILL_ARGS, name, out.data_ptr(), q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
        block_tables.data_ptr(), context_lens.data_ptr(), query_starts.data_ptr(),
        0 if workspace is None else workspace.data_ptr(),
        0 if err_word is None else err_word.data_ptr(), _stream_now(stream, cur), nb,
        0 if workspace is None else workspace.nbytes, _CODES[dt], bs, hk, d, mb, rows,
        tokens, hq, scale)


def prefill_step(out, q, k_new, v_new, slot_mapping, k_pool, v_pool, block_tables, context_lens,
                 query_starts, scale, workspace, *, cos_sin=None, positions=None, sections=None,
                 interleaved: bool = False, q_weight=None, k_weight=None, eps: float = 1e-6,
                 q_rotated=None, err_word=None, stream=None):
    """One layer's prompt step: the new tokens' k and v into the pools, then
    their attention.  With ``cos_sin`` and ``positions`` np_rope_append rotates
    (and, with weights, normalises) q and k on the way: the rotated q goes to
    ``q_rotated`` (default: back into q, which must then be dense).  Without
    them np_kv_append copies k_new and v_new as they are.  What either call
    refuses is refused before the first launch: nothing is written, and the
    step may be called again."""
    if cos_sin is None and any(x is not None for x in (positions, sections, q_weight, k_weight,
                                                       q_rotated)):
        raise ValueError("prefill_step: positions, sections, weights and q_rotated need cos_sin")
    qr = q if q_rotated is None else q_rotated
    attend = _prefill_args(out, qr, k_pool, v_pool, block_tables, context_lens, query_starts, scale,
                           workspace, err_word, stream)
    st = load().np_paged_prefill_check(attend)
    if st != NP_OK:
        raise NPError(st, "np_paged_prefill")
    if cos_sin is not None:
        np_rope_append(qr, q, k_new, v_new, slot_mapping, k_pool, v_pool, cos_sin, positions,
                       sections, interleaved, q_weight, k_weight, eps, err_word, stream)
    else:
        np_kv_append(k_pool, v_pool, k_new, v_new, slot_mapping, err_word, stream)
    _launch_prefill(attend)


# ------------------------------------------------------- the cache in 8 bits --
# np_block_map_args, np_kv_append_q8_args and np_read_q8_args (np_paged.h)
_MAP_ARGS = struct.Struct("@11Pq4i")
_APPEND_Q8_ARGS = struct.Struct("@9P3q6i")
_READ_Q8_ARGS = struct.Struct("@12P2q10if")

_FORMS = {torch.float8_e4m3fn: NP_E4M3, torch.int8: NP_INT8}


def q8_pools(num_blocks, block_size, kv_heads, head_dim, form=torch.float8_e4m3fn, device="cuda"):
    """(k_pool, v_pool, k_scale, v_scale) of an empty 8-bit cache: pools
    [num_blocks, block_size, kv_heads, head_dim] of torch.float8_e4m3fn or torch.int8, and a
    power-of-two fp32 scale per block and kv head.  An element stands for code * scale."""
    if form not in _FORMS:
        raise TypeError(f"unsupported form {form}; the cache holds float8_e4m3fn or int8")
    pools = [torch.zeros((num_blocks, block_size, kv_heads, head_dim), dtype=torch.uint8,
                         device=device).view(form) for _ in range(2)]
    scales = [torch.zeros((num_blocks, kv_heads), dtype=torch.float32, device=device) for _ in range(2)]
    return (*pools, *scales)


_INT32, _INT64, _FLOAT = torch.int32, torch.int64, torch.float32


def _q8_shape(name, k_pool, v_pool, k_scale, v_scale):
    """(form, blocks, block size, kv heads, head_dim) of a cache, after the checks."""
    dt, shape = k_pool.dtype, k_pool.shape
    form = _FORMS.get(dt)
    if len(shape) == 4 and form is not None and v_pool.dtype is dt and v_pool.shape == shape and \
            k_scale.dtype is _FLOAT and v_scale.dtype is _FLOAT:
        nb, bs, hk, d = shape
        if k_scale.shape == (nb, hk) and v_scale.shape == (nb, hk):
            return form, nb, bs, hk, d
    if k_pool.dim() != 4 or v_pool.shape != k_pool.shape:
        raise ValueError(f"{name}: pools must be [blocks, block_size, kv_heads, head_dim]")
    form = _FORMS.get(k_pool.dtype)
    if form is None or v_pool.dtype is not k_pool.dtype:
        raise TypeError(f"{name}: pools must be float8_e4m3fn or int8, both the same")
    nb, bs, hk, d = k_pool.shape
    if k_scale.dtype is not torch.float32 or v_scale.dtype is not torch.float32 or \
            k_scale.shape != (nb, hk) or v_scale.shape != (nb, hk):
        raise ValueError(f"{name}: scales must be float32 [blocks, kv_heads]")
    return form, nb, bs, hk, d


def np_block_map(block_tables, context_lens, new_lens, free_blocks, free_count, query_starts,
                 slot_mapping, positions, block_size, kept_lens=None, err_word=None, stream=None):
    """One step of a batch's bookkeeping on the GPU (see np_paged.h): every row keeps its first
    min(context_lens, kept_lens) positions (all, without ``kept_lens``) and gets ``new_lens`` more;
    blocks go back to and come from the end of ``free_blocks``.  Updates block_tables, context_lens,
    free_blocks and free_count; writes query_starts, slot_mapping and positions (both None: the
    tables only).

    block_tables int32 [rows, max_blocks]; context_lens, new_lens, kept_lens int32 [rows];
    free_blocks int32 [num_blocks]; free_count int32 [1]; query_starts int32 [rows + 1];
    slot_mapping int64 [tokens], one at least; positions int32 [tokens]."""
    name = "np_block_map"
    shape = block_tables.shape
    lens = context_lens.shape
    n = 0 if slot_mapping is None else slot_mapping.numel()
    cur = _device_now()
    # (one condition: what it refuses is looked at again to say why)
    if not (block_tables.dtype is _INT32 and len(shape) == 2 and
            context_lens.dtype is _INT32 and len(lens) == 1 and lens[0] == shape[0] and
            new_lens.dtype is _INT32 and new_lens.shape == lens and
            free_blocks.dtype is _INT32 and free_blocks.dim() == 1 and
            free_count.dtype is _INT32 and free_count.numel() == 1 and
            query_starts.dtype is _INT32 and query_starts.dim() == 1 and
            query_starts.numel() == shape[0] + 1 and
            block_tables.get_device() == context_lens.get_device() == new_lens.get_device() ==
            free_blocks.get_device() == free_count.get_device() == query_starts.get_device() == cur and
            block_tables.is_contiguous() and context_lens.is_contiguous() and
            new_lens.is_contiguous() and free_blocks.is_contiguous() and
            query_starts.is_contiguous() and
            (kept_lens is None or (kept_lens.dtype is _INT32 and kept_lens.shape == lens and
                                   kept_lens.get_device() == cur and kept_lens.is_contiguous())) and
            (slot_mapping is None or (n > 0 and slot_mapping.dtype is _INT64 and
                                      slot_mapping.dim() == 1 and slot_mapping.get_device() == cur and
                                      slot_mapping.is_contiguous())) and
            (positions is None or (n > 0 and positions.dtype is _INT32 and positions.dim() == 1 and
                                   positions.numel() == n and positions.get_device() == cur and
                                   positions.is_contiguous())) and
            (err_word is None or (err_word.get_device() == cur and err_word.is_contiguous()))):
        _refuse_map(name, cur, block_tables, context_lens, new_lens, free_blocks, free_count,
                    query_starts, slot_mapping, positions, kept_lens, err_word)
    rows, mb = shape
    st = load().np_block_map_packed(_pack(
        _MAP_ARGS, name, block_tables.data_ptr(), context_lens.data_ptr(), new_lens.data_ptr(),
        0 if kept_lens is None else kept_lens.data_ptr(), free_blocks.data_ptr(),
        free_count.data_ptr(), query_starts.data_ptr(),
        0 if slot_mapping is None else slot_mapping.data_ptr(),
        0 if positions is None else positions.data_ptr(),
        0 if err_word is None else err_word.data_ptr(), _stream_now(stream, cur),
        free_blocks.numel(), mb, rows, block_size, n))
    if st != NP_OK:
        raise NPError(st, name)


def _refuse_map(name, cur, block_tables, context_lens, new_lens, free_blocks, free_count,
                query_starts, slot_mapping, positions, kept_lens, err_word) -> None:
    """np_block_map's refusal of its arguments."""
    if block_tables.dtype is not _INT32 or block_tables.dim() != 2:
        raise ValueError(f"{name}: block_tables must be int32 [rows, max_blocks]")
    rows = block_tables.shape[0]
    for t, what in ((context_lens, "context_lens"), (new_lens, "new_lens"), (kept_lens, "kept_lens")):
        if t is not None and (t.dtype is not _INT32 or t.shape != (rows,)):
            raise ValueError(f"{name}: {what} must be int32 [rows]")
    if free_blocks.dtype is not _INT32 or free_blocks.dim() != 1:
        raise ValueError(f"{name}: free_blocks must be int32 [num_blocks]")
    if free_count.dtype is not _INT32 or free_count.numel() != 1:
        raise ValueError(f"{name}: free_count must be one int32")
    if query_starts.dtype is not _INT32 or query_starts.shape != (rows + 1,):
        raise ValueError(f"{name}: query_starts must be int32 [rows + 1]")
    if slot_mapping is not None and (slot_mapping.dtype is not _INT64 or slot_mapping.dim() != 1):
        raise ValueError(f"{name}: slot_mapping must be int64 [tokens]")
    if slot_mapping is not None and slot_mapping.numel() == 0:
        raise ValueError(f"{name}: slot_mapping has room for no tokens; None asks for the tables only")
    if positions is not None and (slot_mapping is None or positions.dtype is not _INT32 or
                                  positions.shape != slot_mapping.shape):
        raise ValueError(f"{name}: positions must be int32 [tokens], beside a slot_mapping")
    _refuse(cur, block_tables=block_tables, context_lens=context_lens, new_lens=new_lens,
            kept_lens=kept_lens, free_blocks=free_blocks, free_count=free_count,
            query_starts=query_starts, slot_mapping=slot_mapping, positions=positions,
            err_word=err_word)


def np_kv_append_q8(k_pool, v_pool, k_scale, v_scale, k_new, v_new, slot_mapping, err_word=None,
                    stream=None):
    """New K/V [T, kv_heads, head_dim] (bf16 or fp32; tokens may be strided) rounded into the 8-bit
    pools at ``slot_mapping`` (int64 [T]), with a power-of-two scale per block and kv head (see
    np_paged.h).  The tokens of a block stand side by side in ``slot_mapping``."""
    name = "np_kv_append_q8"
    form, nb, bs, hk, d = _q8_shape(name, k_pool, v_pool, k_scale, v_scale)
    shape, dt = k_new.shape, k_new.dtype
    if len(shape) != 3 or shape[1] != hk or shape[2] != d or v_new.shape != shape:
        raise ValueError(f"{name}: k_new/v_new must be [tokens, kv_heads, head_dim] of the pools")
    if v_new.dtype is not dt:
        raise ValueError(f"{name}: k_new and v_new must share a dtype")
    n = shape[0]
    if slot_mapping.dtype is not _INT64 or slot_mapping.dim() != 1 or slot_mapping.numel() != n:
        raise ValueError(f"{name}: slot_mapping must be int64 [tokens]")
    cur = _device_now()
    kp, ks = _token_rows(k_new, "k_new", cur, n, hk, d)
    vp, vs = _token_rows(v_new, "v_new", cur, n, hk, d)
    if not (k_pool.get_device() == v_pool.get_device() == k_scale.get_device() ==
            v_scale.get_device() == slot_mapping.get_device() == cur and
            k_pool.is_contiguous() and v_pool.is_contiguous() and k_scale.is_contiguous() and
            v_scale.is_contiguous() and slot_mapping.is_contiguous() and
            (err_word is None or (err_word.get_device() == cur and err_word.is_contiguous()))):
        _refuse(cur, k_pool=k_pool, v_pool=v_pool, k_scale=k_scale, v_scale=v_scale,
                slot_mapping=slot_mapping, err_word=err_word)
    st = load().np_kv_append_q8_packed(_pack(
        _APPEND_Q8_ARGS, name, k_pool.data_ptr(), v_pool.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), kp, vp, slot_mapping.data_ptr(),
        0 if err_word is None else err_word.data_ptr(), _stream_now(stream, cur), nb, ks, vs, form,
        _CODES[dt], bs, hk, d, n))
    if st != NP_OK:
        raise NPError(st, name)


def _read_q8_args(name, out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens,
                  query_starts, scale, workspace, err_word, stream, query_len, tokens) -> bytes:
    """np_read_q8_args after the binding's checks; q's shape is the caller's to check."""
    form, nb, bs, hk, d = _q8_shape(name, k_pool, v_pool, k_scale, v_scale)
    if q.shape[-1] != d:
        raise ValueError(f"{name}: q/pool shape mismatch")
    if out.shape != q.shape or out.dtype is not q.dtype:
        raise ValueError(f"{name}: out must match q")
    if block_tables.dtype is not torch.int32 or block_tables.dim() != 2:
        raise ValueError(f"{name}: block_tables must be int32 [rows, max_blocks]")
    rows, mb = block_tables.shape
    if context_lens.dtype is not torch.int32 or context_lens.shape != (rows,):
        raise ValueError(f"{name}: context_lens must be int32 [rows]")
    if query_starts is not None and (query_starts.dtype is not torch.int32 or
                                     query_starts.shape != (rows + 1,)):
        raise ValueError(f"{name}: query_starts must be int32 [rows + 1]")
    cur = _device_now()
    if not (out.get_device() == q.get_device() == k_pool.get_device() == v_pool.get_device() ==
            k_scale.get_device() == v_scale.get_device() == block_tables.get_device() ==
            context_lens.get_device() == cur and
            (query_starts is None or (query_starts.get_device() == cur and
                                      query_starts.is_contiguous())) and
            (workspace is None or (workspace.get_device() == cur and workspace.is_contiguous())) and
            (err_word is None or (err_word.get_device() == cur and err_word.is_contiguous())) and
            out.is_contiguous() and q.is_contiguous() and k_pool.is_contiguous() and
            v_pool.is_contiguous() and k_scale.is_contiguous() and v_scale.is_contiguous() and
            block_tables.is_contiguous() and context_lens.is_contiguous()):
        _refuse(cur, out=out, q=q, k_pool=k_pool, v_pool=v_pool, k_scale=k_scale, v_scale=v_scale,
                block_tables=block_tables, context_lens=context_lens, query_starts=query_starts,
                workspace=workspace, err_word=err_word)
    return _pack(
        _READ_Q8_ARGS, name, out.data_ptr(), q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
        k_scale.data_ptr(), v_scale.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(),
        0 if query_starts is None else query_starts.data_ptr(),
        0 if workspace is None else workspace.data_ptr(),
        0 if err_word is None else err_word.data_ptr(), _stream_now(stream, cur), nb,
        0 if workspace is None else workspace.nbytes, form, _CODES[q.dtype], bs, hk, d, mb, rows,
        query_len, tokens, q.shape[-2], scale)


def np_paged_decode_q8_workspace_bytes(head_dim) -> int:
    return load().np_paged_decode_q8_workspace_bytes(head_dim)


def decode_q8_workspace(head_dim, device="cuda") -> torch.Tensor:
    """A workspace for np_paged_decode_q8 (its contents need no initialisation)."""
    n = np_paged_decode_q8_workspace_bytes(head_dim)
    if n == 0:
        raise ValueError(f"unsupported head_dim {head_dim}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def np_paged_decode_q8(out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens, scale,
                       workspace, err_word=None, stream=None):
    """The decode read of an 8-bit cache (see np_paged.h): q/out [rows, q_heads, head_dim], or
    [rows, query_len, q_heads, head_dim] (the rows' last query_len positions), bf16 or fp32."""
    _launch_decode_q8(_decode_q8_args(out, q, k_pool, v_pool, k_scale, v_scale, block_tables,
                                      context_lens, scale, workspace, err_word, stream))


def _decode_q8_args(out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens, scale,
                    workspace, err_word, stream) -> bytes:
    name = "np_paged_decode_q8"
    rows, qn, _, _ = _q_shape(q)
    if block_tables.dim() == 2 and block_tables.shape[0] != rows:
        raise ValueError(f"{name}: block_tables must be int32 [rows, max_blocks]")
    return _read_q8_args(name, out, q, k_pool, v_pool, k_scale, v_scale, block_tables,
                         context_lens, None, scale, workspace, err_word, stream, qn, rows * qn)


def _launch_decode_q8(packed: bytes) -> None:
    st = load().np_paged_decode_q8_packed(packed)
    if st != NP_OK:
        raise NPError(st, "np_paged_decode_q8")


def np_paged_prefill_q8(out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens,
                        query_starts, scale, workspace, err_word=None, stream=None):
    """Attention of ragged chunks over an 8-bit cache (see np_paged.h): as np_paged_prefill, with
    np_kv_append_q8's pools and scales; q/out [tokens, q_heads, head_dim] bf16 or fp32."""
    _launch_prefill_q8(_prefill_q8_args(out, q, k_pool, v_pool, k_scale, v_scale, block_tables,
                                        context_lens, query_starts, scale, workspace, err_word,
                                        stream))


def _prefill_q8_args(out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens,
                     query_starts, scale, workspace, err_word, stream) -> bytes:
    name = "np_paged_prefill_q8"
    if q.dim() != 3:
        raise ValueError(f"{name}: q must be [tokens, q_heads, head_dim]")
    if query_starts is None:
        raise ValueError(f"{name}: query_starts must be int32 [rows + 1]")
    return _read_q8_args(name, out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens,
                         query_starts, scale, workspace, err_word, stream, 0, q.shape[0])


def _launch_prefill_q8(packed: bytes) -> None:
    st = load().np_paged_prefill_q8_packed(packed)
    if st != NP_OK:
        raise NPError(st, "np_paged_prefill_q8")


def _flat_tokens(t: torch.Tensor, stream) -> torch.Tensor:
    """``t`` with its first two dims as one.  Where that is no view (a slice of padded rows), a copy
    that is made on ``stream``, and belongs to it: the call reads it there."""
    try:
        return t.view(-1, *t.shape[2:]) if t.numel() else t.flatten(0, 1)
    except RuntimeError:
        pass
    if stream is None:
        return t.flatten(0, 1)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return t.flatten(0, 1)


def decode_step_q8(out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens, scale,
                   workspace, *, k_new=None, v_new=None, slot_mapping=None, err_word=None,
                   stream=None):
    """One decode step of an 8-bit cache: the rows' new K/V ([rows, kv_heads, head_dim], or
    [rows, query_len, kv_heads, head_dim] with slots [rows, query_len]) appended, if given, then
    the read.  What the read refuses is refused before the append."""
    read = _decode_q8_args(out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens,
                           scale, workspace, err_word, stream)
    if k_new is not None:
        st = load().np_paged_decode_q8_check(read)
        if st != NP_OK:
            raise NPError(st, "np_paged_decode_q8")
        if k_new.dim() == 4:
            k_new, v_new = _flat_tokens(k_new, stream), _flat_tokens(v_new, stream)
        if slot_mapping.dim() == 2:
            slot_mapping = _flat_tokens(slot_mapping, stream)
        np_kv_append_q8(k_pool, v_pool, k_scale, v_scale, k_new, v_new, slot_mapping, err_word,
                        stream)
    _launch_decode_q8(read)


def prefill_step_q8(out, q, k_new, v_new, slot_mapping, k_pool, v_pool, k_scale, v_scale,
                    block_tables, context_lens, query_starts, scale, workspace, *, err_word=None,
                    stream=None):
    """One layer's prompt step of an 8-bit cache: the new tokens' k and v rounded into the pools,
    then their attention.  What the attention refuses is refused before the append."""
    attend = _prefill_q8_args(out, q, k_pool, v_pool, k_scale, v_scale, block_tables, context_lens,
                              query_starts, scale, workspace, err_word, stream)
    st = load().np_paged_prefill_q8_check(attend)
    if st != NP_OK:
        raise NPError(st, "np_paged_prefill_q8")
    np_kv_append_q8(k_pool, v_pool, k_scale, v_scale, k_new, v_new, slot_mapping, err_word, stream)
    _launch_prefill_q8(attend)


def np_paged_decode_plan(rows, q_heads, kv_heads, head_dim, block_size, max_blocks_per_row,
                         dtype, num_sms: int = 0) -> int:
    out = _I32(0)
    st = load().np_paged_decode_plan(rows, q_heads, kv_heads, head_dim, block_size,
                                     max_blocks_per_row, _dtype_code(dtype), num_sms,
                                     ctypes.byref(out))
    _check(st, "np_paged_decode_plan")
    return out.value


def np_paged_decode_split_len(block_size, max_blocks_per_row, num_splits) -> int:
    return load().np_paged_decode_split_len(block_size, max_blocks_per_row, num_splits)


def np_paged_decode_workspace_bytes(rows, q_heads, head_dim, num_splits) -> int:
    return load().np_paged_decode_workspace_bytes(rows, q_heads, head_dim, num_splits)


def workspace(rows, q_heads, head_dim, num_splits, device="cuda",
              query_len: int = 1) -> torch.Tensor | None:
    """A workspace of the size the library asks for (None if unsplit).  No
    call needs its contents initialised; zero-filled only to be reproducible."""
    n = np_paged_decode_workspace_bytes(rows * query_len, q_heads, head_dim, num_splits)
    if n == 0:
        return None
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _check_read_args(call, out, q, k_pool, v_pool, block_tables, context_lens):
    rows, qn, q_heads, d = _q_shape(q)
    nb, bs, hk, d2 = k_pool.shape
    if d2 != d or v_pool.shape != k_pool.shape or q.dtype != k_pool.dtype or \
            v_pool.dtype != k_pool.dtype:
        raise ValueError(f"{call}: q/pool shape or dtype mismatch")
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 or \
            block_tables.shape[0] != rows:
        raise ValueError(f"{call}: block_tables must be int32 [rows, max_blocks]")
    if context_lens.dtype != torch.int32 or context_lens.shape != (rows,):
        raise ValueError(f"{call}: context_lens must be int32 [rows]")
    if out is not None and (out.shape != q.shape or out.dtype != q.dtype):
        raise ValueError(f"{call}: out must match q")
    return rows, qn, q_heads, d, nb, bs, hk


def np_paged_decode(out, q, k_pool, v_pool, block_tables, context_lens, scale,
                    num_splits: int = 1, workspace=None, err_word=None, stream=None):
    """The decode read (see np_paged.h).  Writes ``out`` when num_splits == 1.

    q is [rows, q_heads, head_dim] (one query token per row) or
    [rows, query_len, q_heads, head_dim] (the rows' last query_len positions).
    """
    rows, qn, q_heads, d, nb, bs, hk = _check_read_args(
        "np_paged_decode", out, q, k_pool, v_pool, block_tables, context_lens)
    cur = _current_device()
    ws_ptr = _opt(workspace, "workspace", cur)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load().np_paged_decode(
        _opt(out, "out", cur), _dev(q, "q", cur), _dev(k_pool, "k_pool", cur),
        _dev(v_pool, "v_pool", cur), _dtype_code(q.dtype), nb, bs, hk, d,
        _dev(block_tables, "block_tables", cur), block_tables.shape[1],
        _dev(context_lens, "context_lens", cur), rows, qn, q_heads, float(scale), num_splits,
        ws_ptr, ws_bytes, _opt(err_word, "err_word", cur), _stream(stream))
    _check(st, "np_paged_decode")


def np_paged_append_decode(out, q, k_new, v_new, slot_mapping, k_pool, v_pool, block_tables,
                           context_lens, scale, num_splits: int = 1, workspace=None,
                           err_word=None, stream=None):
    """Append each row's new tokens (at its newest positions) and read, in one launch.

    k_new/v_new: [rows, kv_heads, head_dim] (or [rows, query_len, kv_heads,
    head_dim]); slot_mapping: int64 [rows] (or [rows, query_len]).
    """
    st = load().np_paged_append_decode(*_append_decode_args(
        out, q, k_new, v_new, slot_mapping, k_pool, v_pool, block_tables, context_lens, scale,
        num_splits, workspace, err_word, stream))
    _check(st, "np_paged_append_decode")


def _append_decode_args(out, q, k_new, v_new, slot_mapping, k_pool, v_pool, block_tables,
                        context_lens, scale, num_splits, workspace, err_word, stream) -> list:
    """np_paged_append_decode's C arguments, after the checks."""
    rows, qn, q_heads, d, nb, bs, hk = _check_read_args(
        "np_paged_append_decode", out, q, k_pool, v_pool, block_tables, context_lens)
    want = (rows, hk, d) if q.dim() == 3 else (rows, qn, hk, d)
    if tuple(k_new.shape) != want or v_new.shape != k_new.shape or \
            k_new.dtype != k_pool.dtype or v_new.dtype != k_pool.dtype:
        raise ValueError(f"np_paged_append_decode: k_new/v_new must be {list(want)}")
    want_sm = (rows,) if q.dim() == 3 else (rows, qn)
    if slot_mapping.dtype != torch.int64 or tuple(slot_mapping.shape) != want_sm:
        raise ValueError(f"np_paged_append_decode: slot_mapping must be int64 {list(want_sm)}")
    cur = _current_device()
    ws_ptr = _opt(workspace, "workspace", cur)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return [_opt(out, "out", cur), _dev(q, "q", cur), _dev(k_new, "k_new", cur),
            _dev(v_new, "v_new", cur), _dev(slot_mapping, "slot_mapping", cur),
            _dev(k_pool, "k_pool", cur), _dev(v_pool, "v_pool", cur), _dtype_code(q.dtype), nb,
            bs, hk, d, _dev(block_tables, "block_tables", cur), block_tables.shape[1],
            _dev(context_lens, "context_lens", cur), rows, qn, q_heads, float(scale),
            num_splits, ws_ptr, ws_bytes, _opt(err_word, "err_word", cur), _stream(stream)]


def np_paged_decode_reduce(out, workspace, num_splits: int, stream=None):
    """Merge split partials in ``workspace`` into ``out`` ([rows, q_heads, head_dim]
    or [rows, query_len, q_heads, head_dim])."""
    st = load().np_paged_decode_reduce(*_reduce_args(out, workspace, num_splits, stream))
    _check(st, "np_paged_decode_reduce")


def _reduce_args(out, workspace, num_splits, stream) -> list:
    rows, qn, q_heads, d = _q_shape(out, "out")
    ws_bytes = workspace.numel() * workspace.element_size()
    cur = _current_device()
    return [_dev(out, "out", cur), _dtype_code(out.dtype), _dev(workspace, "workspace", cur),
            ws_bytes, rows * qn, q_heads, d, num_splits, _stream(stream)]


class PreparedStep:
    """One decode step -- the fused append and read (np_paged_append_decode)
    and, for a split read, np_paged_decode_reduce -- with its arguments
    checked and converted to C types once.  ``launch()`` re-issues the same
    calls at a fraction of the binding's per-call host cost, for loops that
    run a step again and again on the same buffers (their contents may
    change between launches; their addresses, shapes, the schedule and the
    stream may not).  Arguments as for np_paged_append_decode; ``out`` is
    always the step's output.
    """

    def __init__(self, out, q, k_new, v_new, slot_mapping, k_pool, v_pool, block_tables,
                 context_lens, scale, num_splits: int = 1, workspace=None, err_word=None,
                 stream=None):
        lib = load()
        calls = [("np_paged_append_decode", _append_decode_args(
            out if num_splits <= 1 else None, q, k_new, v_new, slot_mapping, k_pool, v_pool,
            block_tables, context_lens, scale, num_splits, workspace, err_word, stream))]
        if num_splits > 1:
            calls.append(("np_paged_decode_reduce",
                          _reduce_args(out, workspace, num_splits, stream)))
        self._calls = []
        for name, args in calls:
            typed = getattr(lib, name)
            # a second handle to the same symbol, without argtypes: it passes
            # the already-typed arguments through unconverted
            raw = lib._FuncPtr((name, lib))
            raw.restype = ctypes.c_int
            cargs = tuple(t(a) for t, a in zip(typed.argtypes, args))
            self._calls.append((name, raw, cargs))
        self.launches = (2 if num_splits == 0 else 1) + (1 if num_splits > 1 else 0)
        self._refs = (out, q, k_new, v_new, slot_mapping, k_pool, v_pool, block_tables,
                      context_lens, workspace, err_word)  # keep the buffers alive

    def launch(self) -> int:
        """Issue the step; returns the number of library kernels launched."""
        for name, fn, cargs in self._calls:
            st = fn(*cargs)
            if st != NP_OK:
                raise NPError(st, name)
        return self.launches


def np_paged_decode_noalloc(out, q, k_pool, v_pool, block_tables, context_lens, scale,
                            num_splits: int = 1, err_word=None, stream=None):
    """The read plus the split merge with no workspace argument: for callers
    that cannot allocate device memory, the split partials go to a fixed
    NP_NOALLOC_SCRATCH_BYTES array inside the library (see np_paged.h)."""
    if out is None:
        raise ValueError("np_paged_decode_noalloc: out is required")
    rows, qn, q_heads, d, nb, bs, hk = _check_read_args(
        "np_paged_decode_noalloc", out, q, k_pool, v_pool, block_tables, context_lens)
    cur = _current_device()
    st = load().np_paged_decode_noalloc(
        _dev(out, "out", cur), _dev(q, "q", cur), _dev(k_pool, "k_pool", cur),
        _dev(v_pool, "v_pool", cur), _dtype_code(q.dtype), nb, bs, hk, d,
        _dev(block_tables, "block_tables", cur), block_tables.shape[1],
        _dev(context_lens, "context_lens", cur), rows, qn, q_heads, float(scale), num_splits,
        _opt(err_word, "err_word", cur), _stream(stream))
    _check(st, "np_paged_decode_noalloc")


def np_selftest_bounded_wait(err_word, limit_cycles: int, stream=None):
    """Device check of the read's wait-timeout path: a wait that nothing
    completes gives up after ``limit_cycles`` and ORs NP_FLAG_TIMEOUT into
    ``err_word`` (a device int32 tensor); see np_paged.h."""
    st = load().np_selftest_bounded_wait(_dev(err_word, "err_word", _current_device()),
                                         int(limit_cycles), _stream(stream))
    _check(st, "np_selftest_bounded_wait")


def decode_step(out, q, k_pool, v_pool, block_tables, context_lens, scale, *, k_new=None,
                v_new=None, slot_mapping=None, num_splits: int = 1, workspace=None,
                err_word=None, stream=None, fused: bool = True) -> int:
    """One decode step: append (if new K/V given), read, reduce (if split).

    With ``fused`` (the default) and one new token per row, the append runs
    inside the read's launch (np_paged_append_decode); otherwise
    np_kv_append runs first.  Returns the number of library kernels launched.
    """
    launches = 0
    o = out if num_splits <= 1 else None  # 0: the balanced read writes out itself
    if k_new is not None and fused and k_new.shape[0] == q.shape[0] and \
            k_new.dim() == q.dim():
        np_paged_append_decode(o, q, k_new, v_new, slot_mapping, k_pool, v_pool, block_tables,
                               context_lens, scale, num_splits, workspace, err_word, stream)
        launches += (2 if num_splits == 0 else 1) if q.shape[0] > 0 else 0  # + the merge
    else:
        if k_new is not None:
            np_kv_append(k_pool, v_pool, k_new, v_new, slot_mapping, err_word, stream)
            launches += 1 if k_new.shape[0] > 0 else 0
        np_paged_decode(o, q, k_pool, v_pool, block_tables, context_lens, scale, num_splits,
                        workspace, err_word, stream)
        launches += (2 if num_splits == 0 else 1) if q.shape[0] > 0 else 0
    if num_splits > 1:
        np_paged_decode_reduce(out, workspace, num_splits, stream)
        launches += 1 if q.shape[0] > 0 else 0
    return launches


def default_scale(head_dim: int) -> float:
    return 1.0 / math.sqrt(head_dim)
