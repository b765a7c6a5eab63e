"""ctypes binding of libcsa2.so (the CSA2 C ABI declared in include/csa2.h).

Argument marshalling only: every function checks tensor devices, dtypes and
contiguity, passes ``data_ptr()`` values and the CUDA stream handle, and
raises on a non-zero status. All arithmetic runs in the CUDA library. There
is no CPU fallback: importing this module fails if the library is missing.

The ``csa2_*`` functions take caller-allocated output tensors, like the C
ABI. The short-named helpers below them allocate outputs and workspaces with
torch (device memory plumbing) and call the same entry points.
"""

from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa2.so")

IDX_HEADS = 32
IDX_DIM = 128
HEADS = 64
HEAD_DIM = 512
TOPK = 512
SWA = 128
POOL_BLOCK = 8
POOL_BLOCKS = 2048
CAP_ALIGN = 128
MAX_TOPK = 4096
MIN_PAGE = 16
MAX_ROPE_DIM = 128
MAX_BEAMS = 64
MAX_BEAM_K = 64
FP4_FORMATS = {"e8m0": 0, "e4m3": 1}  # scales of packed weights: E8M0 per 32 inputs, E4M3 per 16

STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported shape", -3: "misaligned",
          -4: "CUDA error", -5: "device wait timed out", -6: "workspace", -7: "device rejected input",
          -8: "needs more than the static scratch buffer"}
TOPK_STATIC_SCRATCH_BYTES = 32 << 20


class Csa2Error(RuntimeError):
    def __init__(self, name, rc):
        super().__init__(f"{name} failed with status {rc} ({STATUS.get(rc, 'unknown')})")
        self.status = rc


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"CSA2 CUDA library not built ({LIB_PATH} missing); run "
            "`python -c \"import __graft_entry__ as g; g.build()\"` first")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sig = {
        "csa2_version": (ctypes.c_int, []),
        "csa2_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "csa2_get_last_error": (ctypes.c_int, [vp, ctypes.POINTER(ctypes.c_int)]),
        "csa2_quant_mxfp4": (ctypes.c_int, [vp, i64, i32, vp, vp, vp]),
        "csa2_dequant_mxfp4": (ctypes.c_int, [vp, vp, i64, i32, vp, vp]),
        "csa2_pack_kv_fp4": (ctypes.c_int, [vp, i64, vp, vp, vp]),
        "csa2_unpack_kv_fp4": (ctypes.c_int, [vp, vp, i64, vp, vp]),
        "csa2_pack_fp8_e4m3": (ctypes.c_int, [vp, i64, vp, vp]),
        "csa2_unpack_fp8_e4m3": (ctypes.c_int, [vp, i64, vp, vp]),
        "csa2_kv_append": (ctypes.c_int, [vp, vp, i32, i32, vp, vp, vp, vp, i64, vp, vp, vp]),
        "csa2_index_score": (ctypes.c_int, [vp, vp, vp, i32, vp, vp, i64, vp, vp, i64, vp, vp]),
        "csa2_index_score_claimed": (ctypes.c_int, [vp, vp, vp, i32, vp, vp, i64, vp, i64, vp, vp, vp]),
        "csa2_topk_workspace_size": (sz, [i32, i64, i32]),
        "csa2_topk": (ctypes.c_int, [vp, i32, i64, vp, vp, i32, vp, vp, sz, vp]),
        "csa2_topk_static": (ctypes.c_int, [vp, i32, i64, vp, vp, i32, vp, vp]),
        "csa2_block_pool_workspace_size": (sz, [i32, i64, i32, i32]),
        "csa2_block_pool": (ctypes.c_int, [vp, i32, i64, vp, i32, i32, vp, vp, sz, vp]),
        "csa2_block_max": (ctypes.c_int, [vp, i32, i64, vp, i32, vp, vp]),
        "csa2_topk_candidates": (ctypes.c_int, [vp, i32, i64, vp, vp, i32, i64, vp, vp]),
        "csa2_topk_merge_workspace_size": (sz, [i32, i32, i32, i32]),
        "csa2_topk_merge": (ctypes.c_int, [vp, i32, i32, i32, i32, vp, vp, sz, vp]),
        "csa2_shard_positions": (ctypes.c_int, [vp, i32, i32, i64, i64, vp, vp]),
        "csa2_shard_pool": (ctypes.c_int, [vp, i32, i32, i32, i64, i64, vp, vp, vp]),
        "csa2_attn_merge": (ctypes.c_int, [vp, vp, i32, i32, vp, vp, vp, vp]),
        "csa2_index_topk_workspace_size": (sz, [i32, i64, i32, i32]),
        "csa2_index_topk": (ctypes.c_int, [vp, vp, vp, i32, vp, vp, i64, vp, vp, i64, i32, vp, i32, vp,
                                           vp, sz, vp]),
        "csa2_index_topk_bf16": (ctypes.c_int, [vp, vp, i32, vp, vp, i64, vp, vp, i64, i32, vp, i32, vp, vp, sz,
                                                vp]),
        "csa2_prefill_index_score": (ctypes.c_int, [vp, vp, vp, i32, vp, vp, i64, i64, vp, vp]),
        "csa2_prefill_index_score_compressed": (ctypes.c_int, [vp, vp, vp, i32, vp, vp, i64, i64, i32, vp, vp]),
        "csa2_compress_kv": (ctypes.c_int, [vp, vp, vp, i64, i32, vp, vp, vp, vp]),
        "csa2_sparse_attn_workspace_size": (sz, [i32, i32, i32]),
        "csa2_sparse_attn_kernel_launches": (ctypes.c_int, [i32, i32, i32]),
        "csa2_sparse_attn_decode": (ctypes.c_int, [vp, i32, i32, vp, vp, i64, vp, vp, i32, vp, i32, f32,
                                                   vp, vp, vp, vp, sz, vp]),
        "csa2_sparse_attn_reuse": (ctypes.c_int, [vp, i32, i32, vp, vp, i64, vp, vp, i32, vp, i32, f32,
                                                  vp, vp, vp, vp, sz, vp]),
        "csa2_sparse_attn_prefill": (ctypes.c_int, [vp, i32, vp, vp, i64, vp, i32, vp, i32, f32, vp, vp,
                                                    vp, vp, sz, vp]),
        "csa2_sparse_attn_prefill_replay": (ctypes.c_int, [vp, i32, vp, vp, i64, vp, i32, vp, i32, i32, f32, vp,
                                                           vp, vp, vp, sz, vp]),
        "csa2_rope": (ctypes.c_int, [vp, i64, i32, i32, vp, i64, i32, vp, i32, i32, vp, vp]),
        "csa2_paged_kv_append": (ctypes.c_int, [vp, vp, i32, vp, i32, vp, i64, i32, vp, i32, vp, vp, vp, vp, i64, i32,
                                                vp, i32, vp, vp, vp]),
        "csa2_paged_index_score": (ctypes.c_int, [vp, vp, vp, i32, vp, vp, i64, i32, vp, i32, vp, i64, vp, vp, vp]),
        "csa2_paged_sparse_attn_workspace_size": (sz, [i32, i32, i32, i32]),
        "csa2_paged_sparse_attn_decode": (ctypes.c_int, [vp, i32, i32, vp, vp, i64, i32, vp, i32, vp, vp, i32, vp, i32,
                                                         f32, vp, vp, vp, vp, sz, vp]),
        "csa2_paged_attn_workspace_size": (sz, [i32, i32]),
        "csa2_paged_attn": (ctypes.c_int, [vp, i32, vp, i32, vp, vp, i64, i32, vp, i32, vp, i32, f32, vp, vp, vp, vp,
                                           sz, vp]),
        "csa2_fp4_weights_size": (sz, [i32, i32, i32]),
        "csa2_fp4_weights": (ctypes.c_int, [vp, vp, i32, i32, i32, vp, vp]),
        "csa2_fp4_linear_workspace_size": (sz, [i32, i32, i32]),
        "csa2_fp4_linear": (ctypes.c_int, [vp, i32, vp, i32, i32, i32, f32, vp, vp, vp, sz, vp]),
        "csa2_beam_select_workspace_size": (sz, [i32, i32, i32, i32]),
        "csa2_beam_select": (ctypes.c_int, [vp, i32, i32, i32, i32, i64, vp, i32, vp, vp, vp, vp, vp, sz, vp]),
        "csa2_paged_reorder": (ctypes.c_int, [vp, vp, i32, vp, vp, vp, vp, i32, i64, i32, vp, i32, i32, vp, vp, vp, vp]),
        "csa2_reorder_rows": (ctypes.c_int, [vp, i64, i64, vp, i32, vp, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()

EXPORTED = [n for n in dir(_lib) if n.startswith("csa2_")]


def lib():
    return _lib


# ---- marshalling helpers -----------------------------------------------------

def _p(t):
    return None if t is None else t.data_ptr()


# the current stream's handle without a Stream object (0.4 us instead of 3), where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# the current device of a process that has a CUDA tensor (0.06 us instead of 0.2)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _s(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _stream_on(stream, dev):
    """_s for a call whose device is known to be the current one."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _s(stream)


def _req(t, dtype, name, allow_none=False):
    if t is None:
        if allow_none:
            return
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _call(name, *args):
    rc = getattr(_lib, name)(*args)
    if rc != 0:
        raise Csa2Error(name, rc)


def csa2_version() -> int:
    return _lib.csa2_version()


def csa2_get_last_error(stream=None) -> int:
    st = ctypes.c_int(0)
    _call("csa2_get_last_error", _s(stream), ctypes.byref(st))
    return st.value


# ---- codecs ------------------------------------------------------------------

def csa2_quant_mxfp4(x, data, e8m0, stream=None):
    _req(x, torch.bfloat16, "x"); _req(data, torch.uint8, "data"); _req(e8m0, torch.uint8, "e8m0")
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    assert data.numel() == rows * cols // 2 and e8m0.numel() == rows * cols // 32
    _call("csa2_quant_mxfp4", _p(x), rows, cols, _p(data), _p(e8m0), _s(stream))


def csa2_dequant_mxfp4(data, e8m0, out, stream=None):
    _req(data, torch.uint8, "data"); _req(e8m0, torch.uint8, "e8m0"); _req(out, torch.float32, "out")
    cols = out.shape[-1]
    rows = out.numel() // cols
    _call("csa2_dequant_mxfp4", _p(data), _p(e8m0), rows, cols, _p(out), _s(stream))


def csa2_pack_kv_fp4(x, kv_data, kv_scale, stream=None):
    _req(x, torch.bfloat16, "x"); _req(kv_data, torch.uint8, "kv_data"); _req(kv_scale, torch.uint8, "kv_scale")
    n = x.numel() // HEAD_DIM
    assert kv_data.numel() == n * 256 and kv_scale.numel() == n * 32
    _call("csa2_pack_kv_fp4", _p(x), n, _p(kv_data), _p(kv_scale), _s(stream))


def csa2_unpack_kv_fp4(kv_data, kv_scale, out, stream=None):
    _req(kv_data, torch.uint8, "kv_data"); _req(kv_scale, torch.uint8, "kv_scale"); _req(out, torch.bfloat16, "out")
    n = out.numel() // HEAD_DIM
    _call("csa2_unpack_kv_fp4", _p(kv_data), _p(kv_scale), n, _p(out), _s(stream))


def csa2_pack_fp8_e4m3(x, out, stream=None):
    _req(x, torch.bfloat16, "x"); _req(out, torch.uint8, "out")
    assert out.numel() == x.numel()
    _call("csa2_pack_fp8_e4m3", _p(x), x.numel(), _p(out), _s(stream))


def csa2_unpack_fp8_e4m3(inp, out, stream=None):
    _req(inp, torch.uint8, "in"); _req(out, torch.bfloat16, "out")
    _call("csa2_unpack_fp8_e4m3", _p(inp), inp.numel(), _p(out), _s(stream))


def csa2_kv_append(kv, ik, kv_data, kv_scale, ik_data, ik_scale, n_visible, n_visible_out=None, stream=None):
    """kv [B,T,512] bf16 (RoPE'd latents), ik [B,T,128] bf16 -> entries at
    n_visible[b] + t of the planes [B,cap,...]; n_visible_out (may be n_visible)."""
    _req(kv, torch.bfloat16, "kv"); _req(ik, torch.bfloat16, "ik")
    for t, n in ((kv_data, "kv_data"), (kv_scale, "kv_scale"), (ik_data, "ik_data"), (ik_scale, "ik_scale")):
        _req(t, torch.uint8, n)
    _req(n_visible, torch.int32, "n_visible"); _req(n_visible_out, torch.int32, "n_visible_out", allow_none=True)
    B, T = kv.shape[0], kv.shape[1]
    _call("csa2_kv_append", _p(kv), _p(ik), B, T, _p(kv_data), _p(kv_scale), _p(ik_data), _p(ik_scale),
          kv_data.shape[1], _p(n_visible), _p(n_visible_out), _s(stream))


def csa2_compress_kv(c, z, bias, m, kv_data, kv_scale, out=None, stream=None):
    """c, z [n_tokens,512] bf16, bias [m,512] fp32 -> entries [n_tokens/m] packed
    into kv_data [.,256] / kv_scale [.,32]; out [n_tokens/m,512] bf16 (optional)."""
    _req(c, torch.bfloat16, "c"); _req(z, torch.bfloat16, "z"); _req(bias, torch.float32, "bias")
    _req(kv_data, torch.uint8, "kv_data"); _req(kv_scale, torch.uint8, "kv_scale")
    _req(out, torch.bfloat16, "out", allow_none=True)
    n_tokens = c.numel() // 512
    n_out = n_tokens // int(m) if int(m) > 0 else 0
    if (z.numel() != c.numel() or bias.numel() < int(m) * 512 or kv_data.numel() < n_out * 256
            or kv_scale.numel() < n_out * 32 or (out is not None and out.numel() < n_out * 512)):
        raise ValueError("csa2_compress_kv: z must match c, bias holds m x 512, and the outputs hold n_tokens / m entries")
    _call("csa2_compress_kv", _p(c), _p(z), _p(bias), n_tokens, int(m), _p(kv_data), _p(kv_scale), _p(out),
          _s(stream))


# ---- indexer, pool, Top-K -----------------------------------------------------

def csa2_index_score(q_data, q_e8m0, w, ik_data, ik_scale, n_visible, scores, positions=None, stream=None):
    """q_data [B,32,64], q_e8m0 [B,32,4], w [B,32]; ik planes [B,cap,64] / [B,cap,4];
    n_visible [B] int32; positions [B,n_pos] or None; scores [B,n_pos] fp32 (out)."""
    for t, n in ((q_data, "q_data"), (q_e8m0, "q_e8m0"), (ik_data, "ik_data"), (ik_scale, "ik_scale")):
        _req(t, torch.uint8, n)
    _req(w, torch.float32, "w"); _req(n_visible, torch.int32, "n_visible"); _req(scores, torch.float32, "scores")
    _req(positions, torch.int32, "positions", allow_none=True)
    B, cap = ik_data.shape[0], ik_data.shape[1]
    n_pos = scores.shape[1]
    _call("csa2_index_score", _p(q_data), _p(q_e8m0), _p(w), B, _p(ik_data), _p(ik_scale), cap,
          _p(n_visible), _p(positions), n_pos, _p(scores), _s(stream))


def csa2_index_score_claimed(q_data, q_e8m0, w, ik_data, ik_scale, n_visible, scores, tile_counters, stream=None):
    """As csa2_index_score without positions; tile_counters [2*B] int32, zero
    before the first call and left zero by every call."""
    for t, n in ((q_data, "q_data"), (q_e8m0, "q_e8m0"), (ik_data, "ik_data"), (ik_scale, "ik_scale")):
        _req(t, torch.uint8, n)
    _req(w, torch.float32, "w"); _req(n_visible, torch.int32, "n_visible"); _req(scores, torch.float32, "scores")
    _req(tile_counters, torch.int32, "tile_counters")
    B, cap = ik_data.shape[0], ik_data.shape[1]
    n_pos = scores.shape[1]
    if tile_counters.numel() < 2 * B:
        raise ValueError("tile_counters needs 2 * B int32")
    _call("csa2_index_score_claimed", _p(q_data), _p(q_e8m0), _p(w), B, _p(ik_data), _p(ik_scale), cap,
          _p(n_visible), n_pos, _p(scores), _p(tile_counters), _s(stream))


def csa2_topk(scores, k, idx, workspace, n_valid=None, positions=None, stream=None):
    _req(scores, torch.float32, "scores"); _req(idx, torch.int32, "idx"); _req(workspace, torch.uint8, "workspace")
    _req(n_valid, torch.int32, "n_valid", allow_none=True); _req(positions, torch.int32, "positions", allow_none=True)
    B, n = scores.shape
    _call("csa2_topk", _p(scores), B, n, _p(n_valid), _p(positions), k, _p(idx), _p(workspace),
          workspace.numel(), _s(stream))


def csa2_topk_static(scores, k, idx, n_valid=None, positions=None, stream=None):
    """csa2_topk without a workspace: for callers that cannot allocate device
    memory. Its scratch is a fixed 32 MiB buffer inside the library, shared by
    all calls (order calls on one stream; overlapping calls race). The first
    call on a device looks the buffer up; make it before any stream capture."""
    _req(scores, torch.float32, "scores"); _req(idx, torch.int32, "idx")
    _req(n_valid, torch.int32, "n_valid", allow_none=True); _req(positions, torch.int32, "positions", allow_none=True)
    B, n = scores.shape
    _call("csa2_topk_static", _p(scores), B, n, _p(n_valid), _p(positions), k, _p(idx), _s(stream))


def csa2_block_pool(scores, n_visible, pool, workspace, block=POOL_BLOCK, n_blocks=POOL_BLOCKS, stream=None):
    _req(scores, torch.float32, "scores"); _req(pool, torch.int32, "pool"); _req(workspace, torch.uint8, "workspace")
    _req(n_visible, torch.int32, "n_visible", allow_none=True)
    B, n = scores.shape
    _call("csa2_block_pool", _p(scores), B, n, _p(n_visible), block, n_blocks, _p(pool), _p(workspace),
          workspace.numel(), _s(stream))


def csa2_index_topk(q_data, q_e8m0, w, ik_data, ik_scale, n_visible, k, idx, workspace, positions=None,
                    n_pos=None, pool_blocks=0, pool=None, stream=None):
    for t, n in ((q_data, "q_data"), (q_e8m0, "q_e8m0"), (ik_data, "ik_data"), (ik_scale, "ik_scale"),
                 (workspace, "workspace")):
        _req(t, torch.uint8, n)
    _req(w, torch.float32, "w"); _req(n_visible, torch.int32, "n_visible"); _req(idx, torch.int32, "idx")
    _req(positions, torch.int32, "positions", allow_none=True); _req(pool, torch.int32, "pool", allow_none=True)
    B, cap = ik_data.shape[0], ik_data.shape[1]
    if n_pos is None:
        n_pos = positions.shape[1] if positions is not None else cap
    _call("csa2_index_topk", _p(q_data), _p(q_e8m0), _p(w), B, _p(ik_data), _p(ik_scale), cap, _p(n_visible),
          _p(positions), n_pos, k, _p(idx), pool_blocks, _p(pool), _p(workspace), workspace.numel(), _s(stream))


def csa2_index_topk_bf16(q, w, ik_data, ik_scale, n_visible, k, idx, workspace, positions=None, n_pos=None,
                         pool_blocks=0, pool=None, stream=None):
    """csa2_index_topk with q [B,32,128] bf16, quantised inside the scan."""
    _req(q, torch.bfloat16, "q")
    for t, n in ((ik_data, "ik_data"), (ik_scale, "ik_scale"), (workspace, "workspace")):
        _req(t, torch.uint8, n)
    _req(w, torch.float32, "w"); _req(n_visible, torch.int32, "n_visible"); _req(idx, torch.int32, "idx")
    _req(positions, torch.int32, "positions", allow_none=True); _req(pool, torch.int32, "pool", allow_none=True)
    B, cap = ik_data.shape[0], ik_data.shape[1]
    if n_pos is None:
        n_pos = positions.shape[1] if positions is not None else cap
    _call("csa2_index_topk_bf16", _p(q), _p(w), B, _p(ik_data), _p(ik_scale), cap, _p(n_visible), _p(positions),
          n_pos, k, _p(idx), pool_blocks, _p(pool), _p(workspace), workspace.numel(), _s(stream))


def csa2_prefill_index_score(q_data, q_e8m0, w, ik_data, ik_scale, p0, scores, stream=None):
    for t, n in ((q_data, "q_data"), (q_e8m0, "q_e8m0"), (ik_data, "ik_data"), (ik_scale, "ik_scale")):
        _req(t, torch.uint8, n)
    _req(w, torch.float32, "w"); _req(scores, torch.float32, "scores")
    T, n_entries = scores.shape
    _call("csa2_prefill_index_score", _p(q_data), _p(q_e8m0), _p(w), T, _p(ik_data), _p(ik_scale), n_entries,
          p0, _p(scores), _s(stream))


def csa2_block_max(scores, bmax, n_visible=None, block=POOL_BLOCK, stream=None):
    """scores [B,n] fp32 -> bmax [B,ceil(n/block)] fp32."""
    _req(scores, torch.float32, "scores"); _req(bmax, torch.float32, "bmax")
    _req(n_visible, torch.int32, "n_visible", allow_none=True)
    B, n = scores.shape
    _call("csa2_block_max", _p(scores), B, n, _p(n_visible), block, _p(bmax), _s(stream))


# ---- context sharding: exchange steps -------------------------------------------

def csa2_topk_candidates(scores, idx, offset, cand, positions=None, stream=None):
    """scores [B,n] fp32, idx [B,k] int32 columns -> cand [B,k,2] int32 pairs
    (fp32 score bits, global position)."""
    _req(scores, torch.float32, "scores"); _req(idx, torch.int32, "idx"); _req(cand, torch.int32, "cand")
    _req(positions, torch.int32, "positions", allow_none=True)
    B, n = scores.shape
    _call("csa2_topk_candidates", _p(scores), B, n, _p(positions), _p(idx), idx.shape[1], int(offset), _p(cand),
          _s(stream))


def csa2_topk_merge(cand, k_out, idx, workspace, stream=None):
    """cand [R,B,k,2] int32 pairs gathered in rank order -> idx [B,k_out] global positions."""
    _req(cand, torch.int32, "cand"); _req(idx, torch.int32, "idx"); _req(workspace, torch.uint8, "workspace")
    R, B, k = cand.shape[0], cand.shape[1], cand.shape[2]
    _call("csa2_topk_merge", _p(cand), R, B, k, k_out, _p(idx), _p(workspace), workspace.numel(), _s(stream))


def csa2_shard_positions(idx, lo, hi, local_idx, stream=None):
    _req(idx, torch.int32, "idx"); _req(local_idx, torch.int32, "local_idx")
    B, k = idx.shape
    _call("csa2_shard_positions", _p(idx), B, k, int(lo), int(hi), _p(local_idx), _s(stream))


def csa2_shard_pool(blocks, lo, hi, pool, n_visible=None, block=POOL_BLOCK, stream=None):
    _req(blocks, torch.int32, "blocks"); _req(pool, torch.int32, "pool")
    _req(n_visible, torch.int32, "n_visible", allow_none=True)
    B, nb = blocks.shape
    _call("csa2_shard_pool", _p(blocks), B, nb, block, int(lo), int(hi), _p(n_visible), _p(pool), _s(stream))


def csa2_attn_merge(parts, lses, out, out_f32=None, lse_out=None, stream=None):
    """parts [R,...,64,512] fp32, lses [R,...,64] fp32 -> out [...,64,512] bf16."""
    _req(parts, torch.float32, "parts"); _req(lses, torch.float32, "lses"); _req(out, torch.bfloat16, "out")
    _req(out_f32, torch.float32, "out_f32", allow_none=True); _req(lse_out, torch.float32, "lse_out", allow_none=True)
    R = parts.shape[0]
    n_q = parts[0].numel() // (HEADS * HEAD_DIM)
    _call("csa2_attn_merge", _p(parts), _p(lses), R, n_q, _p(out), _p(out_f32), _p(lse_out), _s(stream))


def csa2_prefill_index_score_compressed(q_data, q_e8m0, w, ik_data, ik_scale, p0, m, scores, stream=None):
    for t, n in ((q_data, "q_data"), (q_e8m0, "q_e8m0"), (ik_data, "ik_data"), (ik_scale, "ik_scale")):
        _req(t, torch.uint8, n)
    _req(w, torch.float32, "w"); _req(scores, torch.float32, "scores")
    T, n_entries = scores.shape
    _call("csa2_prefill_index_score_compressed", _p(q_data), _p(q_e8m0), _p(w), T, _p(ik_data), _p(ik_scale),
          n_entries, int(p0), int(m), _p(scores), _s(stream))


# ---- attention ------------------------------------------------------------------

def csa2_sparse_attn_kernel_launches(n_queries, k, n_swa) -> int:
    """Kernel launches one attention call makes on the current device."""
    return int(_lib.csa2_sparse_attn_kernel_launches(n_queries, k, n_swa))


def csa2_sparse_attn_decode(q, kv_data, kv_scale, n_visible, idx, swa, out, workspace, out_f32=None, lse=None,
                            sm_scale=1.0, stream=None):
    """q [B,L,64,512] bf16; kv planes [B,cap,256]/[B,cap,32]; idx [B,k]; swa [B,L,n_swa,512] u8."""
    _req(q, torch.bfloat16, "q"); _req(kv_data, torch.uint8, "kv_data"); _req(kv_scale, torch.uint8, "kv_scale")
    _req(n_visible, torch.int32, "n_visible"); _req(idx, torch.int32, "idx"); _req(out, torch.bfloat16, "out")
    _req(workspace, torch.uint8, "workspace"); _req(swa, torch.uint8, "swa", allow_none=True)
    _req(out_f32, torch.float32, "out_f32", allow_none=True); _req(lse, torch.float32, "lse", allow_none=True)
    B, L = q.shape[0], q.shape[1]
    cap = kv_data.shape[1]
    k = idx.shape[1]
    n_swa = swa.shape[2] if swa is not None else 0
    _call("csa2_sparse_attn_decode", _p(q), B, L, _p(kv_data), _p(kv_scale), cap, _p(n_visible), _p(idx), k,
          _p(swa), n_swa, float(sm_scale), _p(out), _p(out_f32), _p(lse), _p(workspace), workspace.numel(),
          _s(stream))


def csa2_sparse_attn_reuse(q, kv_data, kv_scale, n_visible, idx, swa, out, workspace, out_f32=None, lse=None,
                           sm_scale=1.0, stream=None):
    """As csa2_sparse_attn_decode, with each selected tile gathered once for a
    pair of the L Reuse layers (bit-identical results)."""
    _req(q, torch.bfloat16, "q"); _req(kv_data, torch.uint8, "kv_data"); _req(kv_scale, torch.uint8, "kv_scale")
    _req(n_visible, torch.int32, "n_visible"); _req(idx, torch.int32, "idx"); _req(out, torch.bfloat16, "out")
    _req(workspace, torch.uint8, "workspace"); _req(swa, torch.uint8, "swa", allow_none=True)
    _req(out_f32, torch.float32, "out_f32", allow_none=True); _req(lse, torch.float32, "lse", allow_none=True)
    B, L = q.shape[0], q.shape[1]
    cap = kv_data.shape[1]
    k = idx.shape[1]
    n_swa = swa.shape[2] if swa is not None else 0
    _call("csa2_sparse_attn_reuse", _p(q), B, L, _p(kv_data), _p(kv_scale), cap, _p(n_visible), _p(idx), k,
          _p(swa), n_swa, float(sm_scale), _p(out), _p(out_f32), _p(lse), _p(workspace), workspace.numel(),
          _s(stream))


def csa2_sparse_attn_prefill(q, kv_data, kv_scale, idx, swa, n_swa, out, workspace, out_f32=None, lse=None,
                             sm_scale=1.0, stream=None):
    """q [T,64,512] bf16; kv planes [n_entries,256]/[n_entries,32]; idx [T,k];
    swa [T+n_swa-1,512] u8 (query t uses rows t..t+n_swa-1)."""
    _req(q, torch.bfloat16, "q"); _req(kv_data, torch.uint8, "kv_data"); _req(kv_scale, torch.uint8, "kv_scale")
    _req(idx, torch.int32, "idx"); _req(out, torch.bfloat16, "out"); _req(workspace, torch.uint8, "workspace")
    _req(swa, torch.uint8, "swa", allow_none=True)
    _req(out_f32, torch.float32, "out_f32", allow_none=True); _req(lse, torch.float32, "lse", allow_none=True)
    T = q.shape[0]
    n_entries = kv_data.shape[0]
    k = idx.shape[1]
    _call("csa2_sparse_attn_prefill", _p(q), T, _p(kv_data), _p(kv_scale), n_entries, _p(idx), k, _p(swa), n_swa,
          float(sm_scale), _p(out), _p(out_f32), _p(lse), _p(workspace), workspace.numel(), _s(stream))


def csa2_sparse_attn_prefill_replay(q, kv_data, kv_scale, idx, swa, n_swa, replay_row, out, workspace, out_f32=None,
                                    lse=None, sm_scale=1.0, stream=None):
    """csa2_sparse_attn_prefill with the Bounded-Replay cut: query t uses swa
    rows max(t, replay_row) .. t + n_swa - 1."""
    _req(q, torch.bfloat16, "q"); _req(kv_data, torch.uint8, "kv_data"); _req(kv_scale, torch.uint8, "kv_scale")
    _req(idx, torch.int32, "idx"); _req(out, torch.bfloat16, "out"); _req(workspace, torch.uint8, "workspace")
    _req(swa, torch.uint8, "swa", allow_none=True)
    _req(out_f32, torch.float32, "out_f32", allow_none=True); _req(lse, torch.float32, "lse", allow_none=True)
    T = q.shape[0]
    n_entries = kv_data.shape[0]
    k = idx.shape[1]
    _call("csa2_sparse_attn_prefill_replay", _p(q), T, _p(kv_data), _p(kv_scale), n_entries, _p(idx), k, _p(swa),
          n_swa, int(replay_row), float(sm_scale), _p(out), _p(out_f32), _p(lse), _p(workspace), workspace.numel(),
          _s(stream))


# ---- the cache in pages ---------------------------------------------------------
# Planes are [n_pages, page_size, width]; entry e of sequence b is row
# e % page_size of page page_table[b, e // page_size].

# (A decode step makes several of these calls; their checks are written to cost
# little, and say what is wrong only when something is.)
_U8, _I32, _F32 = torch.uint8, torch.int32, torch.float32

def _refuse(t, dtype, name, dev):
    _req(t, dtype, name)
    raise ValueError(f"{name} is on {t.device}, the call's device is cuda:{dev}")


def _take(t, dtype, name, dev):
    """The address of a contiguous tensor of this type on the call's device."""
    if t is not None and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, dtype, name, dev)


def _device(t, name):
    """The device of a call: its first tensor's, which has to be the current one
    (the kernels are launched there)."""
    if t is None or not t.is_cuda or not t.is_contiguous():
        _req(t, t.dtype if t is not None else None, name)
    dev = t.get_device()
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _pool(dev, planes, page_table, n_visible):
    """(addresses of the planes, n_pages, page_size, table, B, max_pages, counts)."""
    at = []
    pages = None
    for t, width, name in planes:
        at.append(_take(t, torch.uint8, name, dev))
        shape = t.shape
        if pages is None and len(shape) == 3:
            pages = shape[0], shape[1]
        if pages is None or shape != (*pages, width):
            raise ValueError(f"{name} must be [n_pages, page_size, {width}] like the other planes")
    table = _take(page_table, torch.int32, "page_table", dev)
    counts = _take(n_visible, torch.int32, "n_visible", dev)
    shape = page_table.shape
    if len(shape) != 2 or n_visible.shape != (shape[0],):
        raise ValueError("page_table must be [B, max_pages] and n_visible [B]")
    return at, pages[0], pages[1], table, shape[0], shape[1], counts


def _shaped(t, dtype, shape, name, dev):
    if t is None or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, dtype, name, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    return t.data_ptr()


def _plain(tensors, dtype, dev):
    """Whether all are contiguous, of this type and on the call's device."""
    for t in tensors:
        if t is None or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
            return False
    return True


def _optional(t, dtype, shape, name, dev):
    return None if t is None else _shaped(t, dtype, shape, name, dev)


def _rope_table(rope, dev):
    at = _take(rope, torch.float32, "rope", dev)
    shape = rope.shape
    if len(shape) != 3 or shape[2] != 2:
        raise ValueError("rope must be [n_rope, rope_dim / 2, 2]")
    return at, shape[0], 2 * shape[1]


def csa2_rope(x, rope, positions, out, interleaved=False, inverse=False, stream=None):
    """x [n_tokens, heads, dim] bf16 -> out (may be x): the last rope_dim
    channels turned by rope [n_rope, rope_dim / 2, 2] fp32 (cos, sin) at
    positions [n_tokens] int32 (None: row t is at position t)."""
    dev = _device(x, "x")
    x_at, out_at = _take(x, torch.bfloat16, "x", dev), _take(out, torch.bfloat16, "out", dev)
    shape = x.shape
    if len(shape) != 3 or out.shape != shape:
        raise ValueError("x must be [n_tokens, heads, dim], out like it")
    rope_at, n_rope, rope_dim = _rope_table(rope, dev)
    n, heads, dim = shape
    _call("csa2_rope", x_at, n, heads, dim, rope_at, n_rope, rope_dim,
          _optional(positions, torch.int32, (n,), "positions", dev), 1 if interleaved else 0, 1 if inverse else 0,
          out_at, _s(stream))


def csa2_paged_kv_append(kv, ik, kv_data, kv_scale, ik_data, ik_scale, page_table, n_visible, n_visible_out=None,
                         cu_tokens=None, rope=None, positions=None, interleaved=False, stream=None):
    """kv [n_tokens, 512], ik [n_tokens, 128] bf16 (before their rotation when a
    rope table is given) -> entries n_visible[b], n_visible[b] + 1, ... of each
    sequence; cu_tokens [B + 1] int32 gives each sequence its rows (None: the
    same number each); n_visible_out may be n_visible."""
    dev = _device(kv, "kv")
    kv_at, ik_at = _take(kv, torch.bfloat16, "kv", dev), _take(ik, torch.bfloat16, "ik", dev)
    n = kv.shape[0] if kv.dim() else 0
    if kv.shape != (n, HEAD_DIM) or ik.shape != (n, IDX_DIM):
        raise ValueError("kv must be [n_tokens, 512] and ik [n_tokens, 128]")
    at, n_pages, page, table, B, max_pages, counts = _pool(
        dev, ((kv_data, 256, "kv_data"), (kv_scale, 32, "kv_scale"), (ik_data, 64, "ik_data"),
              (ik_scale, 4, "ik_scale")), page_table, n_visible)
    rope_at, n_rope, rope_dim = (None, 0, 0) if rope is None else _rope_table(rope, dev)
    if n and rope_dim and not n_rope:
        # (an empty tensor's address is null, and that means: do not rotate)
        raise ValueError("rope holds no position (rope=None takes the rows as they are)")
    _call("csa2_paged_kv_append", kv_at, ik_at, n, _optional(cu_tokens, torch.int32, (B + 1,), "cu_tokens", dev), B,
          rope_at, n_rope, rope_dim, _optional(positions, torch.int32, (n,), "positions", dev), 1 if interleaved else 0,
          *at, n_pages, page, table, max_pages, counts,
          _optional(n_visible_out, torch.int32, (B,), "n_visible_out", dev), _s(stream))


def csa2_paged_index_score(q_data, q_e8m0, w, ik_data, ik_scale, page_table, n_visible, scores, tile_counters=None,
                           stream=None):
    """q_data [B, 32, 64], q_e8m0 [B, 32, 4], w [B, 32]; scores [B, n_pos] fp32
    (out); tile_counters [2 * B] int32 as in csa2_index_score_claimed (None: a
    fixed range of tiles per CTA)."""
    dev = _device(q_data, "q_data")
    q_at, s_at = _take(q_data, torch.uint8, "q_data", dev), _take(q_e8m0, torch.uint8, "q_e8m0", dev)
    w_at, out_at = _take(w, torch.float32, "w", dev), _take(scores, torch.float32, "scores", dev)
    at, n_pages, page, table, B, max_pages, counts = _pool(
        dev, ((ik_data, 64, "ik_data"), (ik_scale, 4, "ik_scale")), page_table, n_visible)
    if q_data.numel() != B * IDX_HEADS * 64 or q_e8m0.numel() != B * IDX_HEADS * 4 or w.numel() != B * IDX_HEADS:
        raise ValueError("q_data, q_e8m0 and w must hold B x 32 heads")
    if scores.dim() != 2 or scores.shape[0] != B:
        raise ValueError("scores must be [B, n_pos]")
    counters = None
    if tile_counters is not None:
        counters = _take(tile_counters, torch.int32, "tile_counters", dev)
        if tile_counters.numel() < 2 * B:
            raise ValueError("tile_counters needs 2 * B int32")
    _call("csa2_paged_index_score", q_at, s_at, w_at, B, *at, n_pages, page, table, max_pages, counts, scores.shape[1],
          out_at, counters, _s(stream))


def csa2_paged_sparse_attn_decode(q, kv_data, kv_scale, page_table, n_visible, idx, swa, out, workspace, out_f32=None,
                                  lse=None, sm_scale=1.0, stream=None):
    """As csa2_sparse_attn_decode, idx [B, k] naming entries of the paged
    sequences; q [B, L, 64, 512] bf16, swa [B, L, n_swa, 512] u8 or None."""
    dev = _device(q, "q")
    q_at, idx_at = _take(q, torch.bfloat16, "q", dev), _take(idx, torch.int32, "idx", dev)
    ws_at = _take(workspace, torch.uint8, "workspace", dev)
    at, n_pages, page, table, B, max_pages, counts = _pool(
        dev, ((kv_data, 256, "kv_data"), (kv_scale, 32, "kv_scale")), page_table, n_visible)
    shape = q.shape
    if len(shape) != 4 or shape[0] != B or shape[2] != HEADS or shape[3] != HEAD_DIM:
        raise ValueError("q must be [B, L, 64, 512]")
    L = shape[1]
    if idx.dim() != 2 or idx.shape[0] != B:
        raise ValueError("idx must be [B, k]")
    swa_at, n_swa = None, 0
    if swa is not None:
        swa_at = _take(swa, torch.uint8, "swa", dev)
        n_swa = swa.shape[2] if swa.dim() == 4 else 0
        if swa.shape != (B, L, n_swa, HEAD_DIM):
            raise ValueError("swa must be [B, L, n_swa, 512]")
    _call("csa2_paged_sparse_attn_decode", q_at, B, L, *at, n_pages, page, table, max_pages, counts, idx_at,
          idx.shape[1], swa_at, n_swa, float(sm_scale), _shaped(out, torch.bfloat16, shape, "out", dev),
          _optional(out_f32, torch.float32, shape, "out_f32", dev),
          _optional(lse, torch.float32, shape[:3], "lse", dev),
          ws_at, workspace.numel(), _s(stream))


def csa2_paged_attn(q, kv_data, kv_scale, page_table, n_visible, out, workspace, cu_q=None, causal=True, out_f32=None,
                    lse=None, sm_scale=1.0, stream=None):
    """Dense attention of q [n_tokens, 64, 512] bf16 over every entry a token
    sees; cu_q [B + 1] int32 gives each sequence its rows (None: the same number
    each); out_f32 [n_tokens, 64, 512] and lse [n_tokens, 64] are optional."""
    dev = _device(q, "q")
    q_at, ws_at = _take(q, torch.bfloat16, "q", dev), _take(workspace, torch.uint8, "workspace", dev)
    at, n_pages, page, table, B, max_pages, counts = _pool(
        dev, ((kv_data, 256, "kv_data"), (kv_scale, 32, "kv_scale")), page_table, n_visible)
    shape = q.shape
    if len(shape) != 3 or shape[1] != HEADS or shape[2] != HEAD_DIM:
        raise ValueError("q must be [n_tokens, 64, 512]")
    _call("csa2_paged_attn", q_at, shape[0], _optional(cu_q, torch.int32, (B + 1,), "cu_q", dev), B, *at, n_pages, page,
          table, max_pages, counts, 1 if causal else 0, float(sm_scale),
          _shaped(out, torch.bfloat16, shape, "out", dev), _optional(out_f32, torch.float32, shape, "out_f32", dev),
          _optional(lse, torch.float32, shape[:2], "lse", dev),
          ws_at, workspace.numel(), _s(stream))


# ---- products with 4-bit weights ---------------------------------------------------

def _format(name):
    if name not in FP4_FORMATS:
        raise ValueError(f"format must be one of {', '.join(FP4_FORMATS)}, got {name!r}")
    return FP4_FORMATS[name]


def csa2_fp4_weights_size(n_out, n_in, format) -> int:
    """Bytes of the laid-out form of an n_out x n_in matrix."""
    return int(_lib.csa2_fp4_weights_size(n_out, n_in, _format(format)))


# bytes of a block of 128 x 256 weights in each format, as the library has them
_BLOCK_BYTES = tuple(int(_lib.csa2_fp4_weights_size(1, 32, kind)) for kind in sorted(FP4_FORMATS.values()))


def _weights_bytes(n_out, n_in, kind):
    """csa2_fp4_weights_size for a product's check of each call, without the call's 0.7 us."""
    return (n_out + 127) // 128 * ((n_in + 255) // 256) * _BLOCK_BYTES[kind]


def csa2_fp4_weights(data, scale, weights, format, stream=None):
    """data [n_out, n_in / 2] u8 and scale [n_out, n_in / 32 (e8m0) or / 16 (e4m3)]
    u8, as the encoders pack them -> weights (u8, csa2_fp4_weights_size bytes)."""
    dev = _device(data, "data")
    if data.dim() != 2:
        raise ValueError("data must be [n_out, n_in / 2]")
    n_out, n_in = data.shape[0], 2 * data.shape[1]
    scale_at = _shaped(scale, torch.uint8, (n_out, n_in // (16 if format == "e4m3" else 32)), "scale", dev)
    weights_at = _take(weights, torch.uint8, "weights", dev)
    if weights.numel() < csa2_fp4_weights_size(n_out, n_in, format):
        raise ValueError("weights needs csa2_fp4_weights_size(n_out, n_in, format) bytes")
    _call("csa2_fp4_weights", _take(data, torch.uint8, "data", dev), scale_at, n_out, n_in, _format(format), weights_at,
          _s(stream))


def csa2_fp4_linear(x, weights, out, workspace, format, scale=1.0, out_f32=None, stream=None):
    """x [n_tokens, n_in] bf16, weights from csa2_fp4_weights -> out [n_tokens,
    n_out] bf16 = scale * x W^T and / or out_f32, the same in fp32 (either may be
    None, not both)."""
    dev = _device(x, "x")
    if x.dtype is not torch.bfloat16:
        _req(x, torch.bfloat16, "x")
    to = out_f32 if out is None else out
    if to is None:
        raise ValueError("out or out_f32 is required")
    x_shape, shape = x.shape, to.shape
    if len(x_shape) != 2 or len(shape) != 2 or shape[0] != x_shape[0]:
        raise ValueError("x must be [n_tokens, n_in], out or out_f32 [n_tokens, n_out]")
    (n, n_in), n_out = x_shape, shape[1]
    kind = _format(format)
    if not _plain((weights, workspace), _U8, dev):
        _take(weights, _U8, "weights", dev)
        _take(workspace, _U8, "workspace", dev)
    if weights.numel() < _weights_bytes(n_out, n_in, kind):
        raise ValueError(f"weights holds fewer than {n_out} x {n_in} weights")
    out_at = None if out is None else _take(out, torch.bfloat16, "out", dev)  # (its shape is the one compared with)
    out32_at = None if out_f32 is None else _shaped(out_f32, torch.float32, shape, "out_f32", dev)
    rc = _lib.csa2_fp4_linear(x.data_ptr(), n, weights.data_ptr(), n_out, n_in, kind, scale, out_at, out32_at,
                              workspace.data_ptr(), workspace.numel(), _stream_on(stream, dev))
    if rc != 0:
        raise Csa2Error("csa2_fp4_linear", rc)


# ---- beam search -------------------------------------------------------------------

def csa2_beam_select(logits, scores, out_scores, out_parents, out_tokens, workspace, lse=None, stream=None):
    """logits [B, W, V] bf16 or fp32 (rows any distance apart, elements adjacent),
    scores [B, W] fp32 or None -> the k best (beam, token) pairs of each sequence:
    out_scores fp32, out_parents (rows b * W + w) and out_tokens int32 [B, k]; lse
    [B, W] fp32 is optional."""
    dev = _device(out_scores, "out_scores")
    if logits is None:
        raise ValueError("logits is required")
    f32 = logits.dtype is torch.float32
    shape, out_shape = logits.shape, out_scores.shape
    if len(shape) != 3 or not (f32 or logits.dtype is torch.bfloat16) or logits.get_device() != dev:
        raise ValueError(f"logits must be [B, W, V] of bf16 or fp32 on the current device, cuda:{dev}")
    B, W, V = shape
    if logits.is_contiguous():
        ld = V
    else:
        at = logits.stride()
        ld = at[1] if W > 1 else at[0] if B > 1 else V
        if (V > 1 and at[2] != 1) or (B > 1 and at[0] != W * ld):
            raise ValueError("logits must have adjacent elements and equally distant rows")
    if len(out_shape) != 2 or out_shape[0] != B:
        raise ValueError("out_scores must be [B, k]")
    k = out_shape[1]
    if not (_plain((out_scores,), _F32, dev) and _plain((out_parents, out_tokens), _I32, dev)
            and out_parents.shape == out_shape == out_tokens.shape):
        _take(out_scores, _F32, "out_scores", dev)
        _shaped(out_parents, _I32, out_shape, "out_parents", dev)
        _shaped(out_tokens, _I32, out_shape, "out_tokens", dev)
    scores_at = None if scores is None else _shaped(scores, _F32, (B, W), "scores", dev)
    lse_at = None if lse is None else _shaped(lse, _F32, (B, W), "lse", dev)
    rc = _lib.csa2_beam_select(logits.data_ptr(), 1 if f32 else 0, B, W, V, ld, scores_at, k, out_scores.data_ptr(),
                               out_parents.data_ptr(), out_tokens.data_ptr(), lse_at,
                               _take(workspace, _U8, "workspace", dev), workspace.numel(), _stream_on(stream, dev))
    if rc != 0:
        raise Csa2Error("csa2_beam_select", rc)


def csa2_paged_reorder(parents, fresh_pages, page_table, n_visible, page_table_out, n_visible_out, kv_data=None,
                       kv_scale=None, ik_data=None, ik_scale=None, stream=None):
    """Row r takes over the entries of row parents[r] [R] int32: full pages shared, a
    partly filled last page copied into fresh_pages[r] for all rows but the first with
    that parent. Planes [n_pages, page, width], or [layers, n_pages, page, width] for
    caches that share the table; page_table [rows, max_pages] -> page_table_out [R,
    max_pages], n_visible [rows] -> n_visible_out [R]."""
    dev = _device(parents, "parents")
    each = parents.shape
    if len(each) != 1:
        raise ValueError("parents must be [R]")
    first = kv_data if kv_data is not None else ik_data
    if first is None or (kv_data is None) != (kv_scale is None) or (ik_data is None) != (ik_scale is None):
        raise ValueError("codes and scales of the latents, of the keys, or of both are required")
    pool = tuple(first.shape)[:-1]
    if len(pool) == 2:
        layers, (n_pages, page) = 1, pool
    elif len(pool) == 3:
        layers, n_pages, page = pool
    else:
        raise ValueError("planes must be [n_pages, page_size, width] or [layers, n_pages, page_size, width]")
    kv_at = kvs_at = ik_at = iks_at = None
    if kv_data is not None:
        if not _plain((kv_data, kv_scale), _U8, dev) or kv_data.shape != (*pool, 256) or kv_scale.shape != (*pool, 32):
            _shaped(kv_data, _U8, (*pool, 256), "kv_data", dev)
            _shaped(kv_scale, _U8, (*pool, 32), "kv_scale", dev)
        kv_at, kvs_at = kv_data.data_ptr(), kv_scale.data_ptr()
    if ik_data is not None:
        if not _plain((ik_data, ik_scale), _U8, dev) or ik_data.shape != (*pool, 64) or ik_scale.shape != (*pool, 4):
            _shaped(ik_data, _U8, (*pool, 64), "ik_data", dev)
            _shaped(ik_scale, _U8, (*pool, 4), "ik_scale", dev)
        ik_at, iks_at = ik_data.data_ptr(), ik_scale.data_ptr()
    if not _plain((parents, fresh_pages, page_table, n_visible, page_table_out, n_visible_out), _I32, dev):
        for t, name in ((parents, "parents"), (fresh_pages, "fresh_pages"), (page_table, "page_table"),
                        (n_visible, "n_visible"), (page_table_out, "page_table_out"), (n_visible_out, "n_visible_out")):
            _take(t, _I32, name, dev)
    shape = page_table.shape
    if len(shape) != 2:
        raise ValueError("page_table must be [rows, max_pages]")
    (R,), (rows, max_pages) = each, shape
    if (fresh_pages.shape != each or n_visible_out.shape != each or n_visible.shape != (rows,)
            or page_table_out.shape != (R, max_pages)):
        raise ValueError("fresh_pages and n_visible_out must be [R], n_visible [rows], page_table_out [R, max_pages]")
    rc = _lib.csa2_paged_reorder(
        parents.data_ptr(), fresh_pages.data_ptr(), R, kv_at, kvs_at, ik_at, iks_at, layers, n_pages, page,
        page_table.data_ptr(), rows, max_pages, n_visible.data_ptr(), page_table_out.data_ptr(),
        n_visible_out.data_ptr(), _stream_on(stream, dev))
    if rc != 0:
        raise Csa2Error("csa2_paged_reorder", rc)


def csa2_reorder_rows(src, parents, dst, stream=None):
    """dst[r] = src[parents[r]]: src [rows, ...], dst [R, ...] of any one type, rows of
    a multiple of 16 bytes; parents [R] int32, -1 leaves a row as it was."""
    dev = _device(src, "src")
    dtype, shape = src.dtype, src.shape
    dst_at, to = _take(dst, dtype, "dst", dev), dst.shape
    if len(shape) < 1 or len(to) < 1 or (shape != to and shape[1:] != to[1:]):
        raise ValueError("src must be [rows, ...] and dst [R, ...] with rows alike")
    rows, R = shape[0], to[0]
    size = dtype.itemsize * (src.numel() // rows if rows else math.prod(shape[1:]))
    rc = _lib.csa2_reorder_rows(src.data_ptr(), rows, size, _shaped(parents, _I32, (R,), "parents", dev), R, dst_at,
                                _stream_on(stream, dev))
    if rc != 0:
        raise Csa2Error("csa2_reorder_rows", rc)


# ---- allocating helpers (torch memory plumbing + the entry points above) --------

def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def quant_mxfp4(x, stream=None):
    rows = x.numel() // x.shape[-1]
    data = torch.empty(*x.shape[:-1], x.shape[-1] // 2, dtype=torch.uint8, device=x.device)
    sc = torch.empty(*x.shape[:-1], x.shape[-1] // 32, dtype=torch.uint8, device=x.device)
    csa2_quant_mxfp4(x, data, sc, stream)
    return data, sc


def pack_kv_fp4(x, stream=None):
    data = torch.empty(*x.shape[:-1], 256, dtype=torch.uint8, device=x.device)
    sc = torch.empty(*x.shape[:-1], 32, dtype=torch.uint8, device=x.device)
    csa2_pack_kv_fp4(x, data, sc, stream)
    return data, sc


def pack_fp8(x, stream=None):
    out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    csa2_pack_fp8_e4m3(x, out, stream)
    return out


def topk_workspace(B, n, k, device="cuda"):
    return _ws(_lib.csa2_topk_workspace_size(B, n, k), device)


def pool_workspace(B, n, block=POOL_BLOCK, n_blocks=POOL_BLOCKS, device="cuda"):
    return _ws(_lib.csa2_block_pool_workspace_size(B, n, block, n_blocks), device)


def index_topk_workspace(B, n_pos, k, pool_blocks=0, device="cuda"):
    return _ws(_lib.csa2_index_topk_workspace_size(B, n_pos, k, pool_blocks), device)


def merge_workspace(R, B, k, k_out, device="cuda"):
    return _ws(_lib.csa2_topk_merge_workspace_size(R, B, k, k_out), device)


def attn_workspace(n_queries, k, n_swa, device="cuda"):
    return _ws(_lib.csa2_sparse_attn_workspace_size(n_queries, k, n_swa), device)


def paged_attn_workspace(n_tokens, B, device="cuda"):
    return _ws(_lib.csa2_paged_attn_workspace_size(n_tokens, B), device)


def paged_sparse_attn_workspace(B, L, k, n_swa, device="cuda"):
    return _ws(_lib.csa2_paged_sparse_attn_workspace_size(B, L, k, n_swa), device)


def fp4_weights(data, scale, format, stream=None):
    """Packed weights laid out for csa2_fp4_linear."""
    weights = torch.empty(csa2_fp4_weights_size(data.shape[0], 2 * data.shape[1], format), dtype=torch.uint8,
                          device=data.device)
    csa2_fp4_weights(data, scale, weights, format, stream)
    return weights


def fp4_linear_workspace(n_tokens, n_in, format, device="cuda"):
    return _ws(_lib.csa2_fp4_linear_workspace_size(n_tokens, n_in, _format(format)), device)


def beam_select_workspace(B, W, V, k, device="cuda"):
    return _ws(_lib.csa2_beam_select_workspace_size(B, W, V, k), device)
