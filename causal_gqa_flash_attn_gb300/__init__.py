"""Causal grouped-query flash attention for GB300 (sm_103a).

A thin ctypes binding of libfa.so (C ABI in include/fa.h). Every function
takes torch tensors that already live on the GPU, checks dtype/contiguity,
passes raw pointers and the current CUDA stream, and raises FAError on a
non-OK status. All arithmetic runs in the library's CUDA kernels; there is no
CPU fallback, and importing this package fails if the library was not built
(run ``python -m causal_gqa_flash_attn_gb300.build`` or
``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libfa.so")

KV_F32 = 0
KV_Q4_0 = 1
KV_F16 = 2
KV_FP8_E4M3 = 3
Q4_SINK_MAX = 8
Q4_RING_ROWS = 256

T_F32, T_F16, T_BF16 = 0, 1, 2
_TYPES = {torch.float32: T_F32, torch.float16: T_F16, torch.bfloat16: T_BF16}

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_CUDA, ERR_DEVICE, ERR_TIMEOUT, ERR_WORKSPACE = range(7)

# Public entry points of include/fa.h with their ctypes signatures.
_P, _I, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_L, _F = ctypes.c_int64, ctypes.c_float
SIGNATURES = {
    "fa_kv_plane_bytes": (_SZ, [_I, _I, _I, _I]),
    "fa_kv_plane_layout": (_I, [_I, _I, _I, _I, _P, _P, _P, _P]),
    "fa_kv_init": (_I, [_P, _I, _I, _I, _I, _I, _I, _I, _P]),
    "fa_kv_scale_offset": (_SZ, [_I, _I, _I, _I]),
    "fa_kv_set_scale": (_I, [_P, _I, _I, _I, _I, _I, ctypes.c_float, _P]),
    "fa_kv_append": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P]),
    "fa_prefill_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "fa_prefill_tile_shape": (_I, [_I, _P, _P]),
    "fa_prefill": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _SZ, _P,
                        _P]),
    "fa_prefill_lse": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _SZ,
                            _P, _P]),
    "fa_merge_attn_states": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "fa_prefill_chunk_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "fa_prefill_chunk_workspace_bytes_for": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "fa_prefill_chunk": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P,
                              _SZ, _P, _P]),
    "fa_decode_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "fa_decode": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _SZ,
                       _P]),
    "fa_decode_combine": (_I, [_P, _P, _I, _I, _I, _I, _P]),
    "fa_decode_noalloc": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                               _P, _P]),
    "fa_page_bytes": (_SZ, [_I, _I, _I]),
    "fa_page_plan": (_I, [_P, _P, _I, _P, _I, _P, _P, _P, _I, _I, _P, _P, _P, _P, _I, _P]),
    "fa_rope_table": (_I, [_P, _P, _I, _P, _I, _I]),
    "fa_rope": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _L, _L, _L, _L, _P, _L, _I, _P, _I,
                     _I, _P]),
    "fa_paged_append": (_I, [_P, _P, _I, _L, _L, _P, _I, _P, _I, _I, _I, _I, _P]),
    "fa_rope_append": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _L, _L, _L, _L, _P, _L, _I, _P,
                            _I, _P, _P, _I, _I, _P]),
    "fa_paged_gather": (_I, [_P, _I, _P, _I, _P, _I, _I, _I, _I, _P, _P, _I, _P]),
    "fa_paged_attn_workspace_bytes": (_SZ, [_I]),
    "fa_paged_attn": (_I, [_P, _P, _P, _I, _L, _L, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I,
                           _I, _I, _I, _F, _P, _SZ, _P]),
    "fa_paged_attn_scored": (_I, [_P, _P, _P, _I, _L, _L, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I,
                                  _I, _I, _I, _I, _F, _F, _P, _P, _SZ, _P]),
    "fa_packed_attn_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "fa_packed_attn": (_I, [_P, _P, _P, _P, _P, _I, _L, _L, _L, _L, _P, _P, _I, _I, _I, _I, _I, _I,
                            _I, _F, _F, _P, _P, _SZ, _P]),
    "fa_packed_attn_grad_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "fa_packed_attn_grad": (_I, [_P] * 9 + [_I] + [_L] * 8 + [_P, _P, _I, _I, _I, _I, _I, _I, _I,
                                                              _F, _F, _P, _P, _SZ, _P]),
    "fa_set_kernel_events": (_I, [_P, _P]),
    "fa_get_device_error": (_I, [_P]),
    "fa_status_string": (ctypes.c_char_p, [_I]),
    "fa_version": (_I, []),
}


class FAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libfa.so; raises ImportError if it was not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libfa.so not built ({LIB_PATH}); run "
                              "python -m causal_gqa_flash_attn_gb300.build")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().fa_status_string(status).decode()


def _check(status: int, what: str):
    if status != OK:
        raise FAError(status, what)


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor | None, dtype, name: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# ------------------------------------------------------------------ planes

def kv_plane_bytes(kv_fmt: int, n_kv_heads: int, max_seq: int, head_dim: int) -> int:
    return int(lib().fa_kv_plane_bytes(kv_fmt, n_kv_heads, max_seq, head_dim))


def kv_plane_layout(kv_fmt: int, n_kv_heads: int, max_seq: int, head_dim: int):
    """(row_bytes, body_offset, sink_offset, ring_offset) of one plane."""
    vals = [ctypes.c_size_t(0) for _ in range(4)]
    _check(lib().fa_kv_plane_layout(kv_fmt, n_kv_heads, max_seq, head_dim,
                                    *[ctypes.byref(v) for v in vals]), "fa_kv_plane_layout")
    return tuple(int(v.value) for v in vals)


def kv_scale_offset(kv_fmt: int, n_kv_heads: int, max_seq: int, head_dim: int) -> int:
    """Byte offset of an fp8 plane's fp32 scale (0 for the other formats)."""
    return int(lib().fa_kv_scale_offset(kv_fmt, n_kv_heads, max_seq, head_dim))


def kv_set_scale(planes, kv_fmt: int, n_kv_heads: int, max_seq: int, head_dim: int,
                 scale: float, stream=None):
    """Set the scale of every fp8 plane in ``planes`` (consecutive planes)."""
    pb = kv_plane_bytes(kv_fmt, n_kv_heads, max_seq, head_dim)
    if pb == 0 or planes.numel() % pb:
        raise ValueError("planes is not a whole number of planes of this geometry")
    _check(lib().fa_kv_set_scale(_dev(planes, torch.uint8, "planes"), planes.numel() // pb,
                                 kv_fmt, n_kv_heads, max_seq, head_dim, float(scale),
                                 _stream(stream)), "fa_kv_set_scale")


def kv_init(planes, kv_fmt: int, n_kv_heads: int, max_seq: int, head_dim: int,
            shadow_sink: int = 0, shadow_win: int = 0, stream=None):
    """fa_kv_init over every plane in ``planes`` (consecutive planes)."""
    pb = kv_plane_bytes(kv_fmt, n_kv_heads, max_seq, head_dim)
    if pb == 0 or planes.numel() % pb:
        raise ValueError("planes is not a whole number of planes of this geometry")
    _check(lib().fa_kv_init(_dev(planes, torch.uint8, "planes"), planes.numel() // pb, kv_fmt,
                            n_kv_heads, max_seq, head_dim, shadow_sink, shadow_win,
                            _stream(stream)), "fa_kv_init")


def alloc_planes(nslots: int, kv_fmt: int, n_kv_heads: int, max_seq: int, head_dim: int,
                 device="cuda", scale: float = 1.0) -> torch.Tensor:
    """nslots consecutive planes as one uint8 tensor, prepared by fa_kv_init;
    fp8 planes get ``scale`` (the per-tensor k_scale or v_scale, 1.0
    uncalibrated)."""
    pb = kv_plane_bytes(kv_fmt, n_kv_heads, max_seq, head_dim)
    if pb == 0:
        raise ValueError("invalid plane geometry")
    planes = torch.empty(nslots * pb, dtype=torch.uint8, device=device)
    kv_init(planes, kv_fmt, n_kv_heads, max_seq, head_dim)
    if kv_fmt == KV_FP8_E4M3 and scale != 1.0:
        kv_set_scale(planes, kv_fmt, n_kv_heads, max_seq, head_dim, scale)
    return planes


def kv_append(k_new, v_new, k_planes, v_planes, pos0, *, n_kv_heads: int, head_dim: int,
              max_seq: int, kv_fmt: int, shadow_sink: int = 0, shadow_win: int = 0,
              stream=None):
    """Append k_new/v_new [nslots][n][n_kv_heads][head_dim] fp32 at pos0[slot] (int32)."""
    nslots, n = k_new.shape[0], k_new.shape[1]
    _check(lib().fa_kv_append(
        _dev(k_new, torch.float32, "k_new"), _dev(v_new, torch.float32, "v_new"),
        _dev(k_planes, torch.uint8, "k_planes"), _dev(v_planes, torch.uint8, "v_planes"),
        _dev(pos0, torch.int32, "pos0"), nslots, n, n_kv_heads, head_dim, max_seq, kv_fmt,
        shadow_sink, shadow_win, _stream(stream)), "fa_kv_append")


# ----------------------------------------------------------------- prefill

def prefill_workspace_bytes(n: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                            kv_fmt: int | None = None, shadow_win: int = 0) -> int:
    """Workspace of fa_prefill; pass kv_fmt and shadow_win to size a Q4_0 cache
    whose shadow window is neither 0 nor the whole ring."""
    if kv_fmt is not None:
        return prefill_chunk_workspace_bytes(0, n, n_q_heads, n_kv_heads, head_dim, kv_fmt,
                                             shadow_win)
    return int(lib().fa_prefill_workspace_bytes(n, n_q_heads, n_kv_heads, head_dim))


def prefill_tile_shape(head_dim: int):
    bq, bk = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().fa_prefill_tile_shape(head_dim, ctypes.byref(bq), ctypes.byref(bk)),
           "fa_prefill_tile_shape")
    return bq.value, bk.value


def prefill(q, k, v, out, n: int, n_q_heads: int, n_kv_heads: int, head_dim: int, sink: int,
            win: int, kv_fmt: int, *, max_seq: int, shadow_sink: int = 0, shadow_win: int = 0,
            workspace: torch.Tensor, tile_map: torch.Tensor | None = None,
            lse: torch.Tensor | None = None, stream=None):
    """fa_prefill (fa_prefill_lse when lse [Hq][n] fp32 is given): q/out
    [n][Hq][hd] fp32, k/v one plane each (uint8 tensors)."""
    args = (_dev(q, torch.float32, "q"), _dev(k, torch.uint8, "k"), _dev(v, torch.uint8, "v"),
            _dev(out, torch.float32, "out"))
    rest = (n, n_q_heads, n_kv_heads, head_dim, sink, win, kv_fmt, max_seq, shadow_sink,
            shadow_win, _dev(workspace, torch.uint8, "workspace"), workspace.numel(),
            _dev(tile_map, torch.uint8, "tile_map"), _stream(stream))
    if lse is None:
        _check(lib().fa_prefill(*args, *rest), "fa_prefill")
    else:
        _check(lib().fa_prefill_lse(*args, _dev(lse, torch.float32, "lse"), *rest),
               "fa_prefill_lse")


def prefill_chunk_workspace_bytes(pos0: int, n: int, n_q_heads: int, n_kv_heads: int,
                                  head_dim: int, kv_fmt: int | None = None,
                                  shadow_win: int = 0) -> int:
    if kv_fmt is not None:
        return int(lib().fa_prefill_chunk_workspace_bytes_for(pos0, n, n_q_heads, n_kv_heads,
                                                              head_dim, kv_fmt, shadow_win))
    return int(lib().fa_prefill_chunk_workspace_bytes(pos0, n, n_q_heads, n_kv_heads, head_dim))


def prefill_chunk(q, k, v, out, pos0: int, n: int, n_q_heads: int, n_kv_heads: int,
                  head_dim: int, sink: int, win: int, kv_fmt: int, *, max_seq: int,
                  shadow_sink: int = 0, shadow_win: int = 0, workspace: torch.Tensor,
                  tile_map: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                  stream=None):
    """fa_prefill_chunk: n queries at positions pos0.. over cache rows 0..pos0+n-1."""
    _check(lib().fa_prefill_chunk(
        _dev(q, torch.float32, "q"), _dev(k, torch.uint8, "k"), _dev(v, torch.uint8, "v"),
        _dev(out, torch.float32, "out"), _dev(lse, torch.float32, "lse"), pos0, n, n_q_heads,
        n_kv_heads, head_dim, sink, win, kv_fmt, max_seq, shadow_sink, shadow_win,
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(),
        _dev(tile_map, torch.uint8, "tile_map"), _stream(stream)), "fa_prefill_chunk")


def merge_attn_states(out, out_lse, prefix, prefix_lse, suffix, suffix_lse, *,
                      prefill_tokens_with_context: int = -1, stream=None):
    """fa_merge_attn_states: outputs [T][H][D] fp32, lses [H][T] fp32 (out_lse may be None)."""
    T, H, D = prefix.shape
    _check(lib().fa_merge_attn_states(
        _dev(out, torch.float32, "out"), _dev(out_lse, torch.float32, "out_lse"),
        _dev(prefix, torch.float32, "prefix"), _dev(prefix_lse, torch.float32, "prefix_lse"),
        _dev(suffix, torch.float32, "suffix"), _dev(suffix_lse, torch.float32, "suffix_lse"),
        T, H, D, prefill_tokens_with_context, _stream(stream)), "fa_merge_attn_states")


# ------------------------------------------------------------------ decode

def decode_workspace_bytes(nslots: int, n_q_heads: int, head_dim: int, max_splits: int) -> int:
    return int(lib().fa_decode_workspace_bytes(nslots, n_q_heads, head_dim, max_splits))


def decode(q, k_planes, v_planes, pos, *, n_q_heads: int, n_kv_heads: int, head_dim: int,
           max_seq: int, sink: int, win: int, kv_fmt: int, shadow_sink: int = 0,
           shadow_win: int = 0, split_keys: int = 256, max_splits: int, workspace: torch.Tensor,
           stream=None):
    """fa_decode: q [nslots][Hq][hd] fp32, pos [nslots] int32 (device)."""
    nslots = q.shape[0]
    _check(lib().fa_decode(
        _dev(q, torch.float32, "q"), _dev(k_planes, torch.uint8, "k_planes"),
        _dev(v_planes, torch.uint8, "v_planes"), _dev(pos, torch.int32, "pos"), nslots,
        n_q_heads, n_kv_heads, head_dim, max_seq, sink, win, kv_fmt, shadow_sink, shadow_win,
        split_keys, max_splits, _dev(workspace, torch.uint8, "workspace"), workspace.numel(),
        _stream(stream)), "fa_decode")


def decode_combine(workspace, out, *, nslots: int, n_q_heads: int, head_dim: int,
                   max_splits: int, stream=None):
    _check(lib().fa_decode_combine(
        _dev(workspace, torch.uint8, "workspace"), _dev(out, torch.float32, "out"), nslots,
        n_q_heads, head_dim, max_splits, _stream(stream)), "fa_decode_combine")


def decode_noalloc(q, k_planes, v_planes, pos, out, *, n_q_heads: int, n_kv_heads: int,
                   head_dim: int, max_seq: int, sink: int, win: int, kv_fmt: int,
                   shadow_sink: int = 0, shadow_win: int = 0, split_keys: int = 256,
                   max_splits: int, stream=None):
    """fa_decode_noalloc: decode + combine into out [nslots][Hq][hd] with the
    partials in the library's fixed device array; for callers that cannot
    allocate device memory. Calls that overlap on the GPU race on that array."""
    nslots = q.shape[0]
    _check(lib().fa_decode_noalloc(
        _dev(q, torch.float32, "q"), _dev(k_planes, torch.uint8, "k_planes"),
        _dev(v_planes, torch.uint8, "v_planes"), _dev(pos, torch.int32, "pos"), nslots,
        n_q_heads, n_kv_heads, head_dim, max_seq, sink, win, kv_fmt, shadow_sink, shadow_win,
        split_keys, max_splits, _dev(out, torch.float32, "out"), _stream(stream)),
        "fa_decode_noalloc")


# ----------------------------------------------------------- paged serving
# These calls are made once per layer of a step that may take microseconds, so
# their checks read each property of a tensor once.

_I32, _U8, _F32 = torch.int32, torch.uint8, torch.float32


def _here(t: torch.Tensor, name: str) -> int:
    """The index of t's device, which must be the current one: calls launch there."""
    here = t.get_device()
    if here < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if here != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current device, "
                         f"cuda:{torch.cuda.current_device()}, got {t.device}")
    return here


def _arg(t: torch.Tensor, name: str, dtype, shape, here: int) -> int:
    """Pointer of a contiguous tensor of this dtype and shape (None: any) on device `here`."""
    if (t.dtype is dtype and t.get_device() == here and (shape is None or t.shape == shape)
            and t.is_contiguous()):
        return t.data_ptr()
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != here:
        raise ValueError(f"{name} must be on cuda:{here}, as the call's other tensors are, "
                         f"got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _heads(t: torch.Tensor, name: str, dtype, shape, here: int):
    """(pointer, token stride) of a [tokens][heads][head_dim] tensor whose tokens
    may lie apart (a slice of a fused projection's output)."""
    tokens, heads, hd = shape
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} of "
                         f"{tuple(t.shape)}")
    if t.get_device() != here:
        raise ValueError(f"{name} must be on cuda:{here}, as the call's other tensors are, "
                         f"got {t.device}")
    step, head, one = t.stride()
    row = heads * hd
    if (one != 1 and hd > 1) or (head != hd and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if step < row:
        if tokens > 1:
            raise ValueError(f"{name}: tokens overlap")
        step = row
    return t.data_ptr(), step


def _type(t: torch.Tensor, name: str) -> int:
    code = _TYPES.get(t.dtype)
    if code is None or t.dim() != 3:
        raise ValueError(f"{name} must be float32, float16 or bfloat16 of shape (tokens, heads, "
                         f"head_dim), got {t.dtype} of {tuple(t.shape)}")
    return code


def _raw_stream(stream, here: int) -> int:
    return torch._C._cuda_getCurrentRawStream(here) if stream is None else _stream(stream)


def page_bytes(n_kv_heads: int, head_dim: int, page_rows: int) -> int:
    return int(lib().fa_page_bytes(n_kv_heads, head_dim, page_rows))


def alloc_pages(n_pages: int, n_kv_heads: int, head_dim: int, page_rows: int,
                device="cuda") -> torch.Tensor:
    """n_pages 4-bit pages as one uint8 tensor (their contents need no preparation)."""
    pb = page_bytes(n_kv_heads, head_dim, page_rows)
    if pb == 0:
        raise ValueError("invalid page geometry")
    return torch.empty(n_pages * pb, dtype=torch.uint8, device=device)


def _pages(pages, n_kv_heads: int, head_dim: int, page_rows: int, here: int):
    pb = lib().fa_page_bytes(n_kv_heads, head_dim, page_rows)
    n = pages.numel()
    if pb == 0 or n == 0 or n % pb:
        raise ValueError("pages is not a whole number of pages of this geometry")
    return _arg(pages, "pages", _U8, None, here), n // pb


def _table(block_table, n_reqs: int, here: int):
    shape = block_table.shape
    if len(shape) != 2 or shape[0] != n_reqs:
        raise ValueError(f"block_table must have shape ({n_reqs}, max_pages), got {tuple(shape)}")
    return _arg(block_table, "block_table", _I32, None, here), shape[1]


def page_plan(cached, fresh, free_ring, ring_state, block_table, ring_state_out, seq_lens,
              cu_fresh, slot_map, positions, *, page_rows: int, stream=None):
    """fa_page_plan: one step's block-table entries, slots and positions from the
    requests' lengths. All int32: cached, fresh, seq_lens [R], block_table
    [R][max_pages], free_ring [n_pages], ring_state [2], ring_state_out [3],
    cu_fresh [R + 1], slot_map and positions [max_tokens]."""
    here = _here(cached, "cached")
    R, T = cached.numel(), slot_map.numel()
    table, max_pages = _table(block_table, R, here)
    _check(lib().fa_page_plan(
        _arg(cached, "cached", _I32, (R,), here), _arg(fresh, "fresh", _I32, (R,), here), R,
        _arg(free_ring, "free_ring", _I32, None, here), free_ring.numel(),
        _arg(ring_state, "ring_state", _I32, (2,), here),
        _arg(ring_state_out, "ring_state_out", _I32, (3,), here), table, max_pages, page_rows,
        _arg(seq_lens, "seq_lens", _I32, (R,), here),
        _arg(cu_fresh, "cu_fresh", _I32, (R + 1,), here),
        _arg(slot_map, "slot_map", _I32, (T,), here),
        _arg(positions, "positions", _I32, (T,), here), T, _raw_stream(stream, here)),
        "fa_page_plan")


def rope_table(inv_freq, sections=None, *, interleaved: bool = False,
               device="cuda") -> torch.Tensor:
    """fa_rope_table on the device, [pairs][4] int32: inv_freq in radians per
    position (any sequence of floats), sections the pairs that turn with each
    position axis (default: all with one axis)."""
    freq = [float(f) for f in inv_freq]
    n = len(freq)
    sections = [n] if sections is None else [int(x) for x in sections]
    host = torch.empty((n, 4), dtype=torch.int32)
    _check(lib().fa_rope_table(host.data_ptr(), (ctypes.c_double * n)(*freq), n,
                               (ctypes.c_int * len(sections))(*sections), len(sections),
                               int(interleaved)), "fa_rope_table")
    return host.to(device)


def rope(q, k, q_out, k_out, positions, table, *, adjacent: bool = False, inverse: bool = False,
         stream=None):
    """fa_rope: q [T][Hq][hd] and k [T][Hkv][hd] (either pair may be None) rotated
    into q_out and k_out (the same tensors: in place) by positions [n_axes][T]
    int32 ([T] for one axis) and a table of rope_table, whose length is half the
    rotated dims."""
    some = q if q is not None else k
    if some is None:
        raise ValueError("rope needs q or k")
    if (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("q and q_out go together, and k and k_out")
    here = _here(some, "q" if q is not None else "k")
    code, dtype = _type(some, "q" if q is not None else "k"), some.dtype
    T, _, hd = some.shape
    qp = qo = kp = ko = None
    qs = qos = ks = kos = hq = hkv = 0
    if q is not None:
        hq = q.shape[1]
        shape = (T, hq, hd)
        qp, qs = _heads(q, "q", dtype, shape, here)
        qo, qos = (qp, qs) if q_out is q else _heads(q_out, "q_out", dtype, shape, here)
    if k is not None:
        _type(k, "k")
        hkv = k.shape[1]
        shape = (T, hkv, hd)
        kp, ks = _heads(k, "k", dtype, shape, here)
        ko, kos = (kp, ks) if k_out is k else _heads(k_out, "k_out", dtype, shape, here)
    where = positions.shape
    axes = where[0] if len(where) == 2 else 1
    if len(where) not in (1, 2) or where[-1] != T:
        raise ValueError(f"positions must have shape (n_axes, {T}), got {tuple(where)}")
    pairs = table.shape[0] if table.dim() else 0
    _check(lib().fa_rope(
        qp, qo, kp, ko, code, T, hq, hkv, hd, 2 * pairs, qs, qos, ks, kos,
        _arg(positions, "positions", _I32, None, here), T, axes,
        _arg(table, "table", _I32, (pairs, 4), here), adjacent, inverse,
        _raw_stream(stream, here)), "fa_rope")


def paged_append(k_new, v_new, slot_map, pages, *, page_rows: int, stream=None):
    """fa_paged_append: k_new, v_new [T][Hkv][hd] into the rows slot_map [T] int32."""
    here = _here(k_new, "k_new")
    code, dtype, shape = _type(k_new, "k_new"), k_new.dtype, k_new.shape
    T, hkv, hd = shape
    kp, ks = _heads(k_new, "k_new", dtype, shape, here)
    vp, vs = _heads(v_new, "v_new", dtype, shape, here)
    pp, n_pages = _pages(pages, hkv, hd, page_rows, here)
    _check(lib().fa_paged_append(kp, vp, code, ks, vs, _arg(slot_map, "slot_map", _I32, (T,), here),
                                 T, pp, n_pages, hkv, hd, page_rows, _raw_stream(stream, here)),
           "fa_paged_append")


def rope_append(q, k_new, v_new, q_out, positions, table, slot_map, pages, *, page_rows: int,
                adjacent: bool = False, stream=None):
    """fa_rope_append: q [T][Hq][hd] (or None) rotated into q_out (the same tensor: in
    place), and k_new, rotated, and v_new [T][Hkv][hd] into the rows slot_map [T] int32;
    positions and table as for rope."""
    here = _here(k_new, "k_new")
    code, dtype, shape = _type(k_new, "k_new"), k_new.dtype, k_new.shape
    T, hkv, hd = shape
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    qp = qo = None
    hq = qs = qos = 0
    if q is not None:
        _type(q, "q")
        hq = q.shape[1]
        qp, qs = _heads(q, "q", dtype, (T, hq, hd), here)
        qo, qos = (qp, qs) if q_out is q else _heads(q_out, "q_out", dtype, (T, hq, hd), here)
    kp, ks = _heads(k_new, "k_new", dtype, shape, here)
    vp, vs = _heads(v_new, "v_new", dtype, shape, here)
    where = positions.shape
    axes = where[0] if len(where) == 2 else 1
    if len(where) not in (1, 2) or where[-1] != T:
        raise ValueError(f"positions must have shape (n_axes, {T}), got {tuple(where)}")
    pairs = table.shape[0] if table.dim() else 0
    pp, n_pages = _pages(pages, hkv, hd, page_rows, here)
    _check(lib().fa_rope_append(
        qp, qo, kp, vp, code, T, hq, hkv, hd, 2 * pairs, qs, qos, ks, vs,
        _arg(positions, "positions", _I32, None, here), T, axes,
        _arg(table, "table", _I32, (pairs, 4), here), adjacent,
        _arg(slot_map, "slot_map", _I32, (T,), here), pp, n_pages, page_rows,
        _raw_stream(stream, here)), "fa_rope_append")


def paged_gather(pages, block_table, seq_lens, k_planes, v_planes, *, n_kv_heads: int,
                 head_dim: int, page_rows: int, max_seq: int, stream=None):
    """fa_paged_gather: rows 0 .. seq_lens[r]-1 of each request into KV_F16 planes
    (uint8, one plane for each request)."""
    here = _here(pages, "pages")
    R = seq_lens.numel()
    pb = lib().fa_kv_plane_bytes(KV_F16, n_kv_heads, max_seq, head_dim)
    if pb == 0 or k_planes.numel() != R * pb or v_planes.numel() != R * pb:
        raise ValueError("k_planes and v_planes must be one KV_F16 plane for each request")
    pp, n_pages = _pages(pages, n_kv_heads, head_dim, page_rows, here)
    table, max_pages = _table(block_table, R, here)
    _check(lib().fa_paged_gather(
        pp, n_pages, table, max_pages, _arg(seq_lens, "seq_lens", _I32, (R,), here), R,
        n_kv_heads, head_dim, page_rows, _arg(k_planes, "k_planes", _U8, None, here),
        _arg(v_planes, "v_planes", _U8, None, here), max_seq, _raw_stream(stream, here)),
        "fa_paged_gather")


def paged_attn_workspace_bytes(head_dim: int) -> int:
    return int(lib().fa_paged_attn_workspace_bytes(head_dim))


def paged_attn(q, out, cu_q, seq_lens, block_table, pages, *, n_kv_heads: int, page_rows: int,
               sink: int = 0, win: int = 0, scale: float = 0.0, lse=None, workspace,
               stream=None, cap: float = 0.0, slopes=None):
    """fa_paged_attn: q, out [T][Hq][hd] (tokens may lie apart), cu_q [R + 1] and
    seq_lens [R] int32, block_table [R][max_pages] int32, lse [Hq][T] fp32 or None;
    with a cap or slopes [Hq] fp32, fa_paged_attn_scored."""
    here = _here(q, "q")
    code, dtype, shape = _type(q, "q"), q.dtype, q.shape
    T, hq, hd = shape
    R = seq_lens.numel()
    qp, qs = _heads(q, "q", dtype, shape, here)
    op, os_ = _heads(out, "out", dtype, shape, here)
    pp, n_pages = _pages(pages, n_kv_heads, hd, page_rows, here)
    table, max_pages = _table(block_table, R, here)
    head = (qp, op, None if lse is None else _arg(lse, "lse", _F32, (hq, T), here), code, qs, os_,
            _arg(cu_q, "cu_q", _I32, (R + 1,), here), _arg(seq_lens, "seq_lens", _I32, (R,), here),
            table, max_pages, pp, n_pages, page_rows, R, T, hq, n_kv_heads, hd, sink, win, scale)
    tail = (_arg(workspace, "workspace", _U8, None, here), workspace.numel(),
            _raw_stream(stream, here))
    if cap == 0.0 and slopes is None:
        _check(lib().fa_paged_attn(*head, *tail), "fa_paged_attn")
    else:
        _check(lib().fa_paged_attn_scored(
            *head, cap, None if slopes is None else _arg(slopes, "slopes", _F32, (hq,), here),
            *tail), "fa_paged_attn_scored")


# -------------------------------------------------------- packed documents

def packed_attn_workspace_bytes(n_docs: int, n_tokens: int, n_q_heads: int, n_kv_heads: int,
                                head_dim: int) -> int:
    return int(lib().fa_packed_attn_workspace_bytes(n_docs, n_tokens, n_q_heads, n_kv_heads,
                                                    head_dim))


def _packed_rule(cu_docs, prefix, slopes, hq: int, here: int):
    """(documents, pointers of cu_docs, prefix and slopes) of a packed call."""
    D = cu_docs.numel() - 1
    if D < 0 or cu_docs.dim() != 1:
        raise ValueError(f"cu_docs must have shape (n_docs + 1,), got {tuple(cu_docs.shape)}")
    return (D, _arg(cu_docs, "cu_docs", _I32, None, here),
            None if prefix is None else _arg(prefix, "prefix", _I32, (D,), here),
            None if slopes is None else _arg(slopes, "slopes", _F32, (hq,), here))


def packed_attn(q, k, v, out, cu_docs, *, prefix=None, sink: int = 0, win: int = 0,
                scale: float = 0.0, cap: float = 0.0, slopes=None, lse=None, workspace,
                stream=None):
    """fa_packed_attn: q, out [T][Hq][hd] and k, v [T][Hkv][hd] float16 or bfloat16
    (tokens may lie apart), cu_docs [docs + 1] int32, prefix [docs] int32 or None,
    slopes [Hq] fp32 or None, lse [Hq][T] fp32 or None."""
    here = _here(q, "q")
    code, dtype, shape = _type(q, "q"), q.dtype, q.shape
    T, hq, hd = shape
    _type(k, "k")
    hkv = k.shape[1]
    qp, qs = _heads(q, "q", dtype, shape, here)
    kp, ks = _heads(k, "k", dtype, (T, hkv, hd), here)
    vp, vs = _heads(v, "v", dtype, (T, hkv, hd), here)
    op, os_ = _heads(out, "out", dtype, shape, here)
    D, cu, pre, sl = _packed_rule(cu_docs, prefix, slopes, hq, here)
    _check(lib().fa_packed_attn(
        qp, kp, vp, op, None if lse is None else _arg(lse, "lse", _F32, (hq, T), here), code, qs,
        ks, vs, os_, cu, pre, D, T, hq, hkv, hd, sink, win, scale, cap, sl,
        _arg(workspace, "workspace", _U8, None, here), workspace.numel(),
        _raw_stream(stream, here)), "fa_packed_attn")


def packed_attn_grad_workspace_bytes(n_docs: int, n_tokens: int, n_q_heads: int, n_kv_heads: int,
                                     head_dim: int) -> int:
    return int(lib().fa_packed_attn_grad_workspace_bytes(n_docs, n_tokens, n_q_heads, n_kv_heads,
                                                         head_dim))


def packed_attn_grad(q, k, v, out, lse, dout, dq, dk, dv, cu_docs, *, prefix=None, sink: int = 0,
                     win: int = 0, scale: float = 0.0, cap: float = 0.0, slopes=None, workspace,
                     stream=None):
    """fa_packed_attn_grad: dq, dk, dv (like q, k, v) from dout (like out), with the
    inputs, out and lse of the packed_attn call and its cu_docs, prefix and scores."""
    here = _here(q, "q")
    code, dtype, shape = _type(q, "q"), q.dtype, q.shape
    T, hq, hd = shape
    _type(k, "k")
    hkv = k.shape[1]
    kv = (T, hkv, hd)
    tensors = (("q", q, shape), ("k", k, kv), ("v", v, kv), ("out", out, shape),
               ("dout", dout, shape), ("dq", dq, shape), ("dk", dk, kv), ("dv", dv, kv))
    (qp, qs), (kp, ks), (vp, vs), (op, os_), (dop, dos), (dqp, dqs), (dkp, dks), (dvp, dvs) = (
        _heads(t, name, dtype, its, here) for name, t, its in tensors)
    D, cu, pre, sl = _packed_rule(cu_docs, prefix, slopes, hq, here)
    _check(lib().fa_packed_attn_grad(
        qp, kp, vp, op, _arg(lse, "lse", _F32, (hq, T), here), dop, dqp, dkp, dvp, code, qs, ks,
        vs, os_, dos, dqs, dks, dvs, cu, pre, D, T, hq, hkv, hd, sink, win, scale, cap, sl,
        _arg(workspace, "workspace", _U8, None, here), workspace.numel(),
        _raw_stream(stream, here)), "fa_packed_attn_grad")


def set_kernel_events(start, stop):
    """Record torch.cuda.Event pair around the next tensor-core prefill /
    split-decode kernels (None, None to stop). Events must have been recorded
    once so that they exist."""
    h = lambda e: None if e is None else int(e.cuda_event)
    _check(lib().fa_set_kernel_events(h(start), h(stop)), "fa_set_kernel_events")


def get_device_error(stream=None) -> int:
    """Synchronise the stream; return (and clear) the device status."""
    return int(lib().fa_get_device_error(_stream(stream)))


def version() -> int:
    return int(lib().fa_version())
