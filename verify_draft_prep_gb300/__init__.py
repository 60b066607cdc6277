"""Python binding of libsd_gb300 (speculative-decoding verify + P-EAGLE draft-batch rebuild).

Argument marshalling only: every call forwards raw device pointers, sizes and the current CUDA
stream of the tensors' device to the C ABI declared in include/sd.h; all arithmetic runs in the
library's sm_103a kernels. There is no fallback: if the shared library is missing or fails to
load, every call raises.

Build the library with ``verify_draft_prep_gb300.build()`` (nvcc, sm_103a).
"""

from __future__ import annotations

import ctypes
import os
import threading

from ._build import LIB as LIB_PATH
from ._build import build

SD_F32_PROBS = 0
SD_BF16_LOGITS = 1
SD_K_MAX = 16
SD_VERIFY_NOALLOC_MAX_B = 4096

SD_ERR_TOKEN_RANGE = 1
SD_ERR_BLOCK_TABLE = 2
SD_ERR_NUM_ACCEPTED = 4
SD_ERR_MAP_RANGE = 8
SD_ERR_ZERO_ROW = 16
SD_ERR_TOTAL_RANGE = 32
SD_ERR_WAIT = 64
SD_ERR_DRAFT_COUNT = 128
SD_ERR_KV_SLOT = 256
SD_ERR_KV_RANGE = 512

SD_ROPE_HALVES = 0
SD_ROPE_NEIGHBOURS = 1
SD_ROPE_PLAIN = 0
SD_ROPE_LINEAR = 1
SD_ROPE_NTK = 2
SD_ROPE_BANDS = 3
SD_ROPE_YARN = 4

SD_CUT_MAX_V = 524224
SD_TOP_MAX = 32
SD_TOP_MAX_V = 33554432

EXPORTED = ["sd_verify", "sd_verify_workspace_bytes", "sd_verify_kernels",
            "sd_verify_noalloc", "sd_draft_sample", "sd_pdraft_prepare_padded",
            "sd_verify_ragged", "sd_pdraft_prepare_ragged", "sd_pdraft_expand", "sd_pdraft_prepare", "sd_hidden_gather", "sd_philox_words", "sd_race_E",
            "sd_race_E_approx_error", "sd_race_E_check", "sd_status_string", "sd_version",
            "sd_verify_prepare", "sd_verify_prepare_workspace_bytes", "sd_verify_prepare_kernels",
            "sd_verify_prepare_ragged", "sd_diag_verify_prepare_withheld",
            "sd_verify_prepare_padded", "sd_kv_write", "sd_kv_read", "sd_kv_attend",
            "sd_kv_attend_workspace_bytes", "sd_token_logprobs", "sd_kv_weights", "sd_kv_evict",
            "sd_rope", "sd_rope_table", "sd_truncate", "sd_sample"]

_lock = threading.Lock()
_lib = None


class SDError(RuntimeError):
    pass


def load():
    """Load libsd_gb300.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise SDError(f"{LIB_PATH} is missing: build it with verify_draft_prep_gb300.build()")
        lib = ctypes.CDLL(LIB_PATH)
        P, i32, i64, u32, u64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_long, ctypes.c_uint32,
                                 ctypes.c_uint64)
        lib.sd_verify.argtypes = [i32, i32, i32, i32, P, i64, P, i64, P, P, u64, u32, P, P, P,
                                  P, P, ctypes.c_size_t, P, P]
        lib.sd_verify.restype = i32
        lib.sd_verify_ragged.argtypes = [i32, i32, i32, i32, P, i64, P, i64, P, P, P, u64, u32, P,
                                         P, P, P, P, ctypes.c_size_t, P, P]
        lib.sd_verify_ragged.restype = i32
        lib.sd_verify_noalloc.argtypes = [i32, i32, i32, i32, P, i64, P, i64, P, P, u64, u32, P,
                                          P, P, P, P, P]
        lib.sd_verify_noalloc.restype = i32
        lib.sd_verify_workspace_bytes.argtypes = [i32, i32, i32, i32]
        lib.sd_verify_workspace_bytes.restype = ctypes.c_size_t
        lib.sd_draft_sample.argtypes = [i32, i32, i32, i32, P, i64, P, u64, u32, P, P, P]
        lib.sd_draft_sample.restype = i32
        lib.sd_verify_kernels.argtypes = [i32, i32, i32, i32]
        lib.sd_verify_kernels.restype = i32
        lib.sd_verify_prepare.argtypes = [i32, i32, i32, i32, P, i64, P, i64, P, P, u64, u32, P,
                                          P, P, P, P, P, i32, i32, ctypes.c_int32, i32, P, P, P,
                                          P, P, P, P, P, P, i32, P, i64, i32, P, P, i64, P,
                                          ctypes.c_size_t, P, P]
        lib.sd_verify_prepare.restype = i32
        lib.sd_diag_verify_prepare_withheld.argtypes = [i32, u32] + lib.sd_verify_prepare.argtypes
        lib.sd_diag_verify_prepare_withheld.restype = i32
        lib.sd_verify_prepare_ragged.argtypes = [i32, i32, i32, i32, P, i64, P, i64, P, P, P, u64,
                                                 u32, P, P, P, P, P, P, i32, i32, ctypes.c_int32,
                                                 i32, P, P, P, P, P, P, P, P, P, i32, P, i64, i32,
                                                 P, P, i64, P, ctypes.c_size_t, P, P]
        lib.sd_verify_prepare_ragged.restype = i32
        lib.sd_verify_prepare_workspace_bytes.argtypes = [i32]
        lib.sd_verify_prepare_workspace_bytes.restype = ctypes.c_size_t
        lib.sd_verify_prepare_kernels.argtypes = [i32, i32, i32, i32, i32]
        lib.sd_verify_prepare_kernels.restype = i32
        lib.sd_pdraft_expand.argtypes = [i32, i32, P, P, P, P, i32, i32, ctypes.c_int32, i32,
                                         P, P, P, P, P, P, P, P, P, P, P]
        lib.sd_pdraft_expand.restype = i32
        lib.sd_pdraft_prepare.argtypes = [i32, i32, P, P, P, P, i32, i32, ctypes.c_int32, i32,
                                          P, P, P, P, P, P, P, P, P, i32, P, i64, i32, P, P, i64,
                                          P, P]
        lib.sd_pdraft_prepare.restype = i32
        lib.sd_pdraft_prepare_ragged.argtypes = [i32, i32, P, P, P, P, P, i32, i32,
                                                 ctypes.c_int32, i32, P, P, P, P, P, P, P, P, P,
                                                 i32, P, i64, i32, P, P, i64, P, P]
        lib.sd_pdraft_prepare_ragged.restype = i32
        lib.sd_pdraft_prepare_padded.argtypes = [i32, i32, P, P, P, P, i32, i32, ctypes.c_int32,
                                                 P, P, P, P, P, P, P, P, i32, P, i64, i32, P, P,
                                                 i64, P, P]
        lib.sd_pdraft_prepare_padded.restype = i32
        lib.sd_verify_prepare_padded.argtypes = [i32, i32, i32, i32, P, i64, P, i64, P, P, u64,
                                                 u32, P, P, P, P, P, P, i32, i32, ctypes.c_int32,
                                                 P, P, P, P, P, P, P, P, i32, P, i64, i32, P, P,
                                                 i64, P, ctypes.c_size_t, P, P]
        lib.sd_verify_prepare_padded.restype = i32
        lib.sd_hidden_gather.argtypes = [i32, i32, P, P, P, i64, i32, P, P, i64, P, P]
        lib.sd_hidden_gather.restype = i32
        lib.sd_philox_words.argtypes = [i32, P, u64, P, P]
        lib.sd_philox_words.restype = i32
        lib.sd_race_E.argtypes = [i32, P, P, P]
        lib.sd_race_E.restype = i32
        lib.sd_race_E_approx_error.argtypes = [u32, u64, P, P]
        lib.sd_race_E_approx_error.restype = i32
        lib.sd_race_E_check.argtypes = [u32, u64, P, P]
        lib.sd_race_E_check.restype = i32
        cache = [P, P, i64, i64, i64, P, P, i32, i32]
        lib.sd_kv_write.argtypes = [i32, i32, i32, P, i64, i64, P, i64, i64, P] + cache + [P, P]
        lib.sd_kv_write.restype = i32
        lib.sd_kv_read.argtypes = [i32, i32, i32, i32] + cache + [P, i32, P, P, P, P, i64, i64,
                                                                  P, P]
        lib.sd_kv_read.restype = i32
        lib.sd_kv_attend.argtypes = [i32, i32, i32, i32, i32, i32, P, i64, i64] + cache + [
            P, i32, P, P, ctypes.c_float, i32, P, i64, i64, P, P, ctypes.c_size_t, P, P]
        lib.sd_kv_attend.restype = i32
        lib.sd_kv_attend_workspace_bytes.argtypes = [i32]
        lib.sd_kv_attend_workspace_bytes.restype = ctypes.c_size_t
        lib.sd_token_logprobs.argtypes = [i32, i32, i32, i32, P, i64, P, P, i32, P, P, P, P, P, P,
                                          P]
        lib.sd_token_logprobs.restype = i32
        f32, f64 = ctypes.c_float, ctypes.c_double
        lib.sd_kv_weights.argtypes = [i32, i32, i32, i32, i32, i32, P, i64, i64, P, P, i64, i64, i64,
                                      P, i32, i32, P, i32, P, P, P, f32, i32, f32, P, P, P, P]
        lib.sd_kv_weights.restype = i32
        lib.sd_kv_evict.argtypes = [i32, i32, i32] + cache + [P, P, i32, P, i32, P, i32, i32, i32, P,
                                                              P, P, P]
        lib.sd_kv_evict.restype = i32
        lib.sd_rope.argtypes = [i32, i32, i32, i32, i32, i32, P, P, f32, i32, P, i64, i64, P, i64,
                                i64, P, i64, i64, P, i64, i64, P]
        lib.sd_rope.restype = i32
        lib.sd_rope_table.argtypes = [i32, f64, i32, f64, f64, f64, f64, P, P]
        lib.sd_rope_table.restype = i32
        rows = [i32, i32, i32, i32, P, i64, P, P, P, P]
        lib.sd_truncate.argtypes = rows + [P, i64, P, P, P]
        lib.sd_truncate.restype = i32
        lib.sd_sample.argtypes = rows + [P, P, P, P, P, P]
        lib.sd_sample.restype = i32
        lib.sd_status_string.argtypes = [i32]
        lib.sd_status_string.restype = ctypes.c_char_p
        lib.sd_version.argtypes = []
        lib.sd_version.restype = i32
        _lib = lib
        return lib


def _check(rc: int, what: str):
    if rc != 0:
        msg = load().sd_status_string(rc).decode()
        raise SDError(f"{what} failed: {msg} ({rc})")


def _ptr(t):
    """Device pointer of a tensor on the GPU, or of a pinned host tensor (page-locked host memory
    is addressable by the GPU: the kernels then read it over the host link)."""
    if t is None:
        return None
    if not (t.is_cuda or t.is_pinned()):
        raise SDError("tensors passed to libsd_gb300 must live on the GPU or in pinned memory")
    return t.data_ptr()


def _device(t):
    """The tensor's GPU, or the current GPU for a pinned host tensor."""
    import torch

    return t.device if t.is_cuda else torch.device("cuda", torch.cuda.current_device())


def _stream(t, stream):
    import torch

    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    # a pinned host tensor has no device of its own: the current device's stream
    return torch.cuda.current_stream(_device(t)).cuda_stream


def _row_stride(t):
    if t.dim() != 2 or t.stride(1) != 1:
        raise SDError("row arrays must be 2-D with contiguous rows")
    return t.stride(0)


_workspaces = {}


def workspace(device, B, K, V, dtype):
    """A zeroed verify workspace for this device, shared by calls that pass none (calls on
    concurrent streams must pass their own)."""
    import torch

    need = load().sd_verify_workspace_bytes(B, K, V, dtype)
    key = torch.device(device)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=key)
        _workspaces[key] = ws
    return ws


def sd_verify(target, draft, drafts, out_tokens, num_accepted, temperature=None, seed=0,
              p_at_draft=None, q_at_draft=None, err=None, stream=None, workspace_buf=None,
              request_base=0):
    """Verify K drafts per request (see include/sd.h).

    target: [B*(K+1), V] float32 probabilities or bfloat16 logits; draft: [B*K, V] same dtype;
    drafts: [B, K] int32; out_tokens: [B, K+1] int32; num_accepted: [B] int32;
    temperature: [B] float32 or None; p_at_draft / q_at_draft: [B, K] float32 or None;
    err: [1] int32 or None; workspace_buf: zeroed uint8 device tensor of at least
    sd_verify_workspace_bytes bytes, or None for this device's shared one; request_base: the
    global request index of local request 0 (a shard of a larger batch).
    """
    import torch

    B, K = drafts.shape
    V = target.shape[1]
    if target.dtype == torch.float32:
        dtype = SD_F32_PROBS
    elif target.dtype == torch.bfloat16:
        dtype = SD_BF16_LOGITS
    else:
        raise SDError("target must be float32 probabilities or bfloat16 logits")
    if draft.dtype != target.dtype or draft.shape[1] != V:
        raise SDError("draft must match target's dtype and vocabulary")
    if target.shape[0] != B * (K + 1) or draft.shape[0] != B * K:
        raise SDError("row counts must be B*(K+1) (target) and B*K (draft)")
    ws = workspace_buf if workspace_buf is not None else workspace(_device(target), B, K, V,
                                                                   dtype)
    rc = load().sd_verify(B, K, V, dtype, _ptr(target), _row_stride(target), _ptr(draft),
                          _row_stride(draft), _ptr(drafts), _ptr(temperature), seed,
                          request_base, _ptr(out_tokens), _ptr(num_accepted), _ptr(p_at_draft),
                          _ptr(q_at_draft), _ptr(ws), ws.numel(), _ptr(err),
                          _stream(target, stream))
    _check(rc, "sd_verify")


def sd_verify_prepare(target, draft, drafts, out_tokens, num_accepted, pos0, block_table,
                      block_size, mask_token_id, input_ids, positions, slot_mapping, hidden_map,
                      is_masked, is_rejected, start_loc, new_token_idx, total_out, target_hidden,
                      h_shared, out_hidden, temperature=None, seed=0, p_at_draft=None,
                      q_at_draft=None, err=None, stream=None, workspace_buf=None,
                      request_base=0, diag_withhold=None):
    """sd_verify then sd_pdraft_prepare on its outputs, in one call (see include/sd.h): arguments
    as for the two calls; workspace_buf: zeroed uint8 device tensor of at least
    sd_verify_prepare_workspace_bytes(B) bytes, or None for this device's shared one.
    diag_withhold: test support, (request, wait_us) for sd_diag_verify_prepare_withheld."""
    import torch

    B, K = drafts.shape
    V = target.shape[1]
    if target.dtype == torch.float32:
        dtype = SD_F32_PROBS
    elif target.dtype == torch.bfloat16:
        dtype = SD_BF16_LOGITS
    else:
        raise SDError("target must be float32 probabilities or bfloat16 logits")
    if draft.dtype != target.dtype or draft.shape[1] != V:
        raise SDError("draft must match target's dtype and vocabulary")
    if target.shape[0] != B * (K + 1) or draft.shape[0] != B * K:
        raise SDError("row counts must be B*(K+1) (target) and B*K (draft)")
    cap, H = out_hidden.shape
    if input_ids.shape[0] != cap:
        raise SDError("out_hidden must have one row per drafter slot")
    ws = workspace_buf if workspace_buf is not None else workspace(_device(target), B, K, V,
                                                                   dtype)
    lib = load()
    fn, pre = lib.sd_verify_prepare, ()
    if diag_withhold is not None:
        fn, pre = lib.sd_diag_verify_prepare_withheld, tuple(diag_withhold)
    rc = fn(
        *pre, B, K, V, dtype, _ptr(target), _row_stride(target), _ptr(draft), _row_stride(draft),
        _ptr(drafts), _ptr(temperature), seed, request_base, _ptr(out_tokens),
        _ptr(num_accepted), _ptr(p_at_draft), _ptr(q_at_draft), _ptr(pos0), _ptr(block_table),
        block_table.shape[1], block_size, mask_token_id, cap, _ptr(input_ids), _ptr(positions),
        _ptr(slot_mapping), _ptr(hidden_map), _ptr(is_masked), _ptr(is_rejected),
        _ptr(start_loc), _ptr(new_token_idx), _ptr(total_out), H, _ptr(target_hidden),
        _row_stride(target_hidden), target_hidden.shape[0], _ptr(h_shared), _ptr(out_hidden),
        _row_stride(out_hidden), _ptr(ws), ws.numel(), _ptr(err), _stream(target, stream))
    _check(rc, "sd_verify_prepare")


def sd_verify_prepare_ragged(target, draft, drafts, cu_drafts, out_tokens, num_accepted, pos0,
                             block_table, block_size, mask_token_id, input_ids, positions,
                             slot_mapping, hidden_map, is_masked, is_rejected, start_loc,
                             new_token_idx, total_out, target_hidden, h_shared, out_hidden,
                             temperature=None, seed=0, p_at_draft=None, q_at_draft=None, err=None,
                             stream=None, workspace_buf=None, request_base=0):
    """sd_verify_ragged then sd_pdraft_prepare_ragged on its outputs, in one call (see
    include/sd.h); shapes as for the two calls (out_tokens [B, K_max+1])."""
    import torch

    B, K1 = out_tokens.shape
    V = target.shape[1]
    if target.dtype == torch.float32:
        dtype = SD_F32_PROBS
    elif target.dtype == torch.bfloat16:
        dtype = SD_BF16_LOGITS
    else:
        raise SDError("target must be float32 probabilities or bfloat16 logits")
    if draft.dtype != target.dtype or cu_drafts.shape[0] != B + 1:
        raise SDError("draft must match target; cu_drafts needs B+1 entries")
    cap, H = out_hidden.shape
    if input_ids.shape[0] != cap:
        raise SDError("out_hidden must have one row per drafter slot")
    ws = workspace_buf if workspace_buf is not None else workspace(_device(target), B, K1 - 1, V,
                                                                   dtype)
    rc = load().sd_verify_prepare_ragged(
        B, K1 - 1, V, dtype, _ptr(target), _row_stride(target), _ptr(draft),
        _row_stride(draft) if draft.shape[0] else V, _ptr(drafts), _ptr(cu_drafts),
        _ptr(temperature), seed, request_base, _ptr(out_tokens), _ptr(num_accepted),
        _ptr(p_at_draft), _ptr(q_at_draft), _ptr(pos0), _ptr(block_table), block_table.shape[1],
        block_size, mask_token_id, cap, _ptr(input_ids), _ptr(positions), _ptr(slot_mapping),
        _ptr(hidden_map), _ptr(is_masked), _ptr(is_rejected), _ptr(start_loc),
        _ptr(new_token_idx), _ptr(total_out), H, _ptr(target_hidden),
        _row_stride(target_hidden), target_hidden.shape[0], _ptr(h_shared), _ptr(out_hidden),
        _row_stride(out_hidden), _ptr(ws), ws.numel(), _ptr(err), _stream(target, stream))
    _check(rc, "sd_verify_prepare_ragged")


def sd_verify_prepare_kernels(B, K, V, dtype, has_temperature):
    """Kernels one sd_verify_prepare call launches (0, 1 or 2)."""
    n = load().sd_verify_prepare_kernels(B, K, V, dtype, int(bool(has_temperature)))
    if n < 0:
        _check(n, "sd_verify_prepare_kernels")
    return n


def sd_verify_ragged(target, draft, drafts, cu_drafts, out_tokens, num_accepted, temperature=None,
                     seed=0, p_at_draft=None, q_at_draft=None, err=None, stream=None,
                     workspace_buf=None, request_base=0):
    """Verify with a draft count per request (see include/sd.h).

    cu_drafts: [B+1] int32 exclusive prefix of the counts; target: [cu[B] + B, V] rows;
    draft: [cu[B], V]; drafts: [cu[B]] int32; out_tokens: [B, K_max+1]; p/q_at: [B, K_max].
    """
    import torch

    B, K1 = out_tokens.shape
    V = target.shape[1]
    if target.dtype == torch.float32:
        dtype = SD_F32_PROBS
    elif target.dtype == torch.bfloat16:
        dtype = SD_BF16_LOGITS
    else:
        raise SDError("target must be float32 probabilities or bfloat16 logits")
    if draft.dtype != target.dtype or cu_drafts.shape[0] != B + 1:
        raise SDError("draft must match target; cu_drafts needs B+1 entries")
    ws = workspace_buf if workspace_buf is not None else workspace(_device(target), B, K1 - 1, V,
                                                                   dtype)
    rc = load().sd_verify_ragged(B, K1 - 1, V, dtype, _ptr(target), _row_stride(target),
                                 _ptr(draft), _row_stride(draft) if draft.shape[0] else V,
                                 _ptr(drafts), _ptr(cu_drafts), _ptr(temperature), seed,
                                 request_base, _ptr(out_tokens), _ptr(num_accepted),
                                 _ptr(p_at_draft), _ptr(q_at_draft), _ptr(ws), ws.numel(),
                                 _ptr(err), _stream(target, stream))
    _check(rc, "sd_verify_ragged")


def sd_verify_kernels(B, V, dtype, has_temperature):
    """How many kernels one sd_verify call with these sizes launches on the current device."""
    n = load().sd_verify_kernels(B, V, dtype, int(bool(has_temperature)))
    if n < 0:
        raise SDError(f"sd_verify_kernels: {load().sd_status_string(n).decode()}")
    return n


def sd_draft_sample(rows, drafts, temperature=None, seed=0, request_base=0, err=None,
                    stream=None):
    """Sample the drafter's K new drafts per request (see include/sd.h).

    rows: [B*K, V] float32 probabilities or bfloat16 logits; drafts: [B, K] int32 (output);
    temperature: [B] float32 or None; request_base: global request index of local request 0.
    """
    import torch

    B, K = drafts.shape
    V = rows.shape[1]
    if rows.dtype == torch.float32:
        dtype = SD_F32_PROBS
    elif rows.dtype == torch.bfloat16:
        dtype = SD_BF16_LOGITS
    else:
        raise SDError("rows must be float32 probabilities or bfloat16 logits")
    if rows.shape[0] != B * K:
        raise SDError("rows must hold B*K rows")
    rc = load().sd_draft_sample(B, K, V, dtype, _ptr(rows), _row_stride(rows), _ptr(temperature),
                                seed, request_base, _ptr(drafts), _ptr(err), _stream(rows, stream))
    _check(rc, "sd_draft_sample")


def sd_pdraft_expand(out_tokens, num_accepted, pos0, block_table, block_size, mask_token_id,
                     input_ids, positions, slot_mapping, hidden_map, is_masked, is_rejected,
                     start_loc, new_token_idx, total_out, err=None, stream=None):
    """Rebuild the drafter batch (see include/sd.h). Outputs have `capacity` = len(input_ids)."""
    B, K1 = out_tokens.shape
    rc = load().sd_pdraft_expand(
        B, K1 - 1, _ptr(out_tokens), _ptr(num_accepted), _ptr(pos0), _ptr(block_table),
        block_table.shape[1], block_size, mask_token_id, input_ids.shape[0], _ptr(input_ids),
        _ptr(positions), _ptr(slot_mapping), _ptr(hidden_map), _ptr(is_masked),
        _ptr(is_rejected), _ptr(start_loc), _ptr(new_token_idx), _ptr(total_out), _ptr(err),
        _stream(start_loc, stream))
    _check(rc, "sd_pdraft_expand")


def sd_pdraft_prepare(out_tokens, num_accepted, pos0, block_table, block_size, mask_token_id,
                      input_ids, positions, slot_mapping, hidden_map, is_masked, is_rejected,
                      start_loc, new_token_idx, total_out, target_hidden, h_shared, out_hidden,
                      err=None, stream=None):
    """sd_pdraft_expand and the hidden-state gather in one launch (see include/sd.h)."""
    B, K1 = out_tokens.shape
    cap, H = out_hidden.shape
    if input_ids.shape[0] != cap:
        raise SDError("out_hidden must have one row per drafter slot")
    rc = load().sd_pdraft_prepare(
        B, K1 - 1, _ptr(out_tokens), _ptr(num_accepted), _ptr(pos0), _ptr(block_table),
        block_table.shape[1], block_size, mask_token_id, cap, _ptr(input_ids), _ptr(positions),
        _ptr(slot_mapping), _ptr(hidden_map), _ptr(is_masked), _ptr(is_rejected),
        _ptr(start_loc), _ptr(new_token_idx), _ptr(total_out), H, _ptr(target_hidden),
        _row_stride(target_hidden), target_hidden.shape[0], _ptr(h_shared), _ptr(out_hidden),
        _row_stride(out_hidden), _ptr(err), _stream(start_loc, stream))
    _check(rc, "sd_pdraft_prepare")


def sd_pdraft_prepare_ragged(out_tokens, num_accepted, cu_drafts, pos0, block_table, block_size,
                             mask_token_id, input_ids, positions, slot_mapping, hidden_map,
                             is_masked, is_rejected, start_loc, new_token_idx, total_out,
                             target_hidden, h_shared, out_hidden, err=None, stream=None):
    """sd_pdraft_prepare with a draft count per request (see include/sd.h)."""
    B, K1 = out_tokens.shape
    cap, H = out_hidden.shape
    if input_ids.shape[0] != cap or cu_drafts.shape[0] != B + 1:
        raise SDError("out_hidden needs one row per drafter slot, cu_drafts B+1 entries")
    rc = load().sd_pdraft_prepare_ragged(
        B, K1 - 1, _ptr(out_tokens), _ptr(num_accepted), _ptr(cu_drafts), _ptr(pos0),
        _ptr(block_table), block_table.shape[1], block_size, mask_token_id, cap, _ptr(input_ids),
        _ptr(positions), _ptr(slot_mapping), _ptr(hidden_map), _ptr(is_masked),
        _ptr(is_rejected), _ptr(start_loc), _ptr(new_token_idx), _ptr(total_out), H,
        _ptr(target_hidden), _row_stride(target_hidden), target_hidden.shape[0], _ptr(h_shared),
        _ptr(out_hidden), _row_stride(out_hidden), _ptr(err), _stream(start_loc, stream))
    _check(rc, "sd_pdraft_prepare_ragged")


def sd_pdraft_prepare_padded(out_tokens, num_accepted, pos0, block_table, block_size,
                             mask_token_id, input_ids, positions, slot_mapping, hidden_map,
                             is_masked, rejected, scatter_map, new_token_idx, target_hidden=None,
                             h_shared=None, out_hidden=None, err=None, stream=None):
    """The drafter batch in fixed rows of 2K slots per request (see include/sd.h); outputs have
    B*2K entries (out_hidden [B*2K, H] bf16, or None for the metadata alone)."""
    B, K1 = out_tokens.shape
    K = K1 - 1
    if input_ids.shape[0] != B * 2 * K:
        raise SDError("padded outputs have B*2K entries")
    H = out_hidden.shape[1] if out_hidden is not None else 1
    n_in = target_hidden.shape[0] if target_hidden is not None else 0
    rc = load().sd_pdraft_prepare_padded(
        B, K, _ptr(out_tokens), _ptr(num_accepted), _ptr(pos0), _ptr(block_table),
        block_table.shape[1], block_size, mask_token_id, _ptr(input_ids), _ptr(positions),
        _ptr(slot_mapping), _ptr(hidden_map), _ptr(is_masked), _ptr(rejected),
        _ptr(scatter_map), _ptr(new_token_idx), H, _ptr(target_hidden),
        _row_stride(target_hidden) if target_hidden is not None else H, n_in, _ptr(h_shared),
        _ptr(out_hidden), _row_stride(out_hidden) if out_hidden is not None else H, _ptr(err),
        _stream(input_ids, stream))
    _check(rc, "sd_pdraft_prepare_padded")


def sd_verify_prepare_padded(target, draft, drafts, out_tokens, num_accepted, pos0, block_table,
                             block_size, mask_token_id, input_ids, positions, slot_mapping,
                             hidden_map, is_masked, rejected, scatter_map, new_token_idx,
                             target_hidden=None, h_shared=None, out_hidden=None, temperature=None,
                             seed=0, p_at_draft=None, q_at_draft=None, err=None, stream=None,
                             workspace_buf=None, request_base=0):
    """sd_verify then sd_pdraft_prepare_padded on its outputs, in one call (see include/sd.h):
    arguments as for the two calls; workspace_buf as for sd_verify."""
    import torch

    B, K = drafts.shape
    V = target.shape[1]
    if target.dtype == torch.float32:
        dtype = SD_F32_PROBS
    elif target.dtype == torch.bfloat16:
        dtype = SD_BF16_LOGITS
    else:
        raise SDError("target must be float32 probabilities or bfloat16 logits")
    if draft.dtype != target.dtype or draft.shape[1] != V:
        raise SDError("draft must match target's dtype and vocabulary")
    if target.shape[0] != B * (K + 1) or draft.shape[0] != B * K:
        raise SDError("row counts must be B*(K+1) (target) and B*K (draft)")
    if input_ids.shape[0] != B * 2 * K:
        raise SDError("padded outputs have B*2K entries")
    H = out_hidden.shape[1] if out_hidden is not None else 1
    n_in = target_hidden.shape[0] if target_hidden is not None else 0
    ws = workspace_buf if workspace_buf is not None else workspace(_device(target), B, K, V,
                                                                   dtype)
    rc = load().sd_verify_prepare_padded(
        B, K, V, dtype, _ptr(target), _row_stride(target), _ptr(draft), _row_stride(draft),
        _ptr(drafts), _ptr(temperature), seed, request_base, _ptr(out_tokens),
        _ptr(num_accepted), _ptr(p_at_draft), _ptr(q_at_draft), _ptr(pos0), _ptr(block_table),
        block_table.shape[1], block_size, mask_token_id, _ptr(input_ids), _ptr(positions),
        _ptr(slot_mapping), _ptr(hidden_map), _ptr(is_masked), _ptr(rejected), _ptr(scatter_map),
        _ptr(new_token_idx), H, _ptr(target_hidden),
        _row_stride(target_hidden) if target_hidden is not None else H, n_in, _ptr(h_shared),
        _ptr(out_hidden), _row_stride(out_hidden) if out_hidden is not None else H, _ptr(ws),
        ws.numel(), _ptr(err), _stream(target, stream))
    _check(rc, "sd_verify_prepare_padded")


def sd_hidden_gather(total_out, hidden_map, target_hidden, h_shared, out_hidden, err=None,
                     stream=None):
    """Gather drafter hidden states (see include/sd.h). bf16 rows."""
    cap, H = out_hidden.shape
    rc = load().sd_hidden_gather(cap, H, _ptr(total_out), _ptr(hidden_map), _ptr(target_hidden),
                                 _row_stride(target_hidden), target_hidden.shape[0],
                                 _ptr(h_shared), _ptr(out_hidden), _row_stride(out_hidden),
                                 _ptr(err), _stream(out_hidden, stream))
    _check(rc, "sd_hidden_gather")


def sd_philox_words(ctr, seed, out, stream=None):
    rc = load().sd_philox_words(ctr.shape[0], _ptr(ctr), seed, _ptr(out), _stream(ctr, stream))
    _check(rc, "sd_philox_words")


def sd_race_E(w, E, stream=None):
    rc = load().sd_race_E(w.shape[0], _ptr(w), _ptr(E), _stream(w, stream))
    _check(rc, "sd_race_E")


def sd_race_E_approx_error(w_begin, count, max_rel, stream=None):
    rc = load().sd_race_E_approx_error(w_begin, count, _ptr(max_rel), _stream(max_rel, stream))
    _check(rc, "sd_race_E_approx_error")


def sd_race_E_check(w_begin, count, counts, stream=None):
    """counts: int64 CUDA tensor [2], zeroed: (words differing from the double path, words that
    took the double path) over [w_begin, w_begin + count)."""
    rc = load().sd_race_E_check(w_begin, count, _ptr(counts), _stream(counts, stream))
    _check(rc, "sd_race_E_check")


_torch = None


def _t():
    """torch, imported once (these calls run every few microseconds)."""
    global _torch
    if _torch is None:
        import torch

        _torch = torch
    return _torch


def _quick():
    """The library, without the lock once it is loaded."""
    return _lib if _lib is not None else load()


def _raw_stream(t, stream):
    """The given stream, or the current one of the tensor's device. (As a bare handle, where torch
    gives one: building its stream object takes longer than the rest of a call's checks.)"""
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    raw = getattr(_t()._C, "_cuda_getCurrentRawStream", None)
    if raw is None or not t.is_cuda:
        return _t().cuda.current_stream(_device(t)).cuda_stream
    return raw(t.get_device())


def _cache_args(k_cache, v_cache, k_scale, v_scale):
    """The cache arguments of the C calls: pointers, strides and sizes of a cache in e4m3 (or its
    bytes as uint8), [num_blocks, block_size, Hkv, D], with scales [num_blocks, Hkv] fp32."""
    torch = _t()
    shape, st = k_cache.shape, k_cache.stride()
    kinds = (torch.float8_e4m3fn, torch.uint8)
    if len(shape) != 4 or st[3] != 1 or k_cache.dtype not in kinds or v_cache.dtype not in kinds:
        raise SDError("a cache is e4m3 (or uint8) [num_blocks, block_size, Hkv, D] with "
                      "contiguous heads")
    if v_cache.shape != shape or v_cache.stride() != st:
        raise SDError("k_cache and v_cache must have the same shape and strides")
    nb, bs, Hkv, _ = shape
    for t in (k_scale, v_scale):
        if t.dtype != torch.float32 or t.shape != (nb, Hkv) or not t.is_contiguous():
            raise SDError("scales must be contiguous float32 [num_blocks, Hkv]")
    # a dimension of one has no stride of its own
    return (_ptr(k_cache), _ptr(v_cache), st[0] if nb > 1 else 16, st[1] if bs > 1 else 16,
            st[2] if Hkv > 1 else 16, _ptr(k_scale), _ptr(v_scale), nb, bs)


def _head_rows(t, Hn, D, what):
    """Strides of bf16 [n, heads, D] rows with contiguous heads."""
    shape = t.shape
    if t.dtype != _t().bfloat16 or len(shape) != 3 or shape[1] != Hn or shape[2] != D:
        raise SDError(f"{what} must be bfloat16 [tokens, {Hn}, {D}] with contiguous heads")
    st = t.stride()
    if st[2] != 1 and shape[0]:
        raise SDError(f"{what} must be bfloat16 [tokens, {Hn}, {D}] with contiguous heads")
    return (st[0] if shape[0] > 1 else 0), (st[1] if Hn > 1 else 0)


def _int32(t, shape, what):
    if t.dtype != _t().int32 or t.shape != shape or not t.is_contiguous():
        raise SDError(f"{what} must be contiguous int32 {list(shape)}")


def _float32(t, shape, what):
    if t.dtype != _t().float32 or t.shape != shape or not t.is_contiguous():
        raise SDError(f"{what} must be contiguous float32 {list(shape)}")


def sd_kv_write(k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, err=None, stream=None):
    """Quantise the K and V of n tokens into the pages that slot_mapping names (see include/sd.h).

    k, v: [n, Hkv, D] bfloat16 (strided: they may be slices of one projection); slot_mapping: [n]
    int32, negative where nothing is written; caches: [num_blocks, block_size, Hkv, D]
    float8_e4m3fn; scales: [num_blocks, Hkv] float32 (zeroed before first use).
    """
    cache = _cache_args(k_cache, v_cache, k_scale, v_scale)
    Hkv, D = k_cache.shape[2:]
    n = k.shape[0]
    if v.shape[0] != n:
        raise SDError("k and v must hold the same tokens")
    _int32(slot_mapping, (n,), "slot_mapping")
    rc = _quick().sd_kv_write(n, Hkv, D, _ptr(k), *_head_rows(k, Hkv, D, "k"), _ptr(v),
                            *_head_rows(v, Hkv, D, "v"), _ptr(slot_mapping), *cache, _ptr(err),
                            _raw_stream(k_cache, stream))
    _check(rc, "sd_kv_write")


def sd_kv_read(k_cache, v_cache, k_scale, v_scale, block_table, cu_tokens, k_out, v_out,
               first_pos=None, err=None, stream=None):
    """Read tokens of every request back as bf16 rows (see include/sd.h).

    block_table: [B, max_blocks] int32; cu_tokens: [B+1] int32, the rows of each request; k_out,
    v_out: [n, Hkv, D] bfloat16 of the same strides; first_pos: [B] int32, the position of each
    request's first row, or None for 0.
    """
    cache = _cache_args(k_cache, v_cache, k_scale, v_scale)
    Hkv, D = k_cache.shape[2:]
    B, mb = block_table.shape
    _int32(block_table, (B, mb), "block_table")
    _int32(cu_tokens, (B + 1,), "cu_tokens")
    if first_pos is not None:
        _int32(first_pos, (B,), "first_pos")
    strides = _head_rows(k_out, Hkv, D, "k_out")
    if v_out.shape != k_out.shape or _head_rows(v_out, Hkv, D, "v_out") != strides:
        raise SDError("k_out and v_out must have the same shape and strides")
    rc = _quick().sd_kv_read(B, k_out.shape[0], Hkv, D, *cache, _ptr(block_table), mb,
                           _ptr(cu_tokens), _ptr(first_pos), _ptr(k_out), _ptr(v_out), *strides,
                           _ptr(err), _raw_stream(k_cache, stream))
    _check(rc, "sd_kv_read")


def attend_workspace(device, D=128):
    """A scratch buffer of sd_kv_attend on this device, for heads of up to D values."""
    return _t().empty(sd_kv_attend_workspace_bytes(D), dtype=_t().uint8, device=device)


_attend_bytes = {}  # by D


def _take_scratch(t, size, stream):
    """Device memory for one call on one stream, and what gives it back: the allocator hands it out again
    in that stream's order, and to a captured graph from the graph's own pool, so that no two calls
    meet in it. (As a bare address, where torch gives one: a tensor takes 4 us more of each call.)"""
    torch = _t()
    take = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
    give = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)
    if take is not None and give is not None and t.is_cuda:
        return take(size, stream), give
    device = _device(t)
    if device.type != "cuda":
        held = torch.empty(size, dtype=torch.uint8)
    else:
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
            held = torch.empty(size, dtype=torch.uint8, device=device)
    return held.data_ptr(), lambda at, held=held: None


def sd_kv_attend_workspace_bytes(D):
    """Bytes of scratch that sd_kv_attend needs for heads of D values."""
    return _quick().sd_kv_attend_workspace_bytes(D)


def sd_kv_attend(q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens, cu_q, out, lse=None,
                 max_q=None, sm_scale=None, causal=True, workspace_buf=None, err=None,
                 stream=None):
    """Attention of each request's new tokens to its cached ones (see include/sd.h).

    q, out: [n, Hq, D] bfloat16; ctx_lens: [B] int32, tokens in the cache, the new ones included;
    cu_q: [B+1] int32, the query tokens of each request; lse: [n, Hq] float32 or None; max_q: the
    most query tokens of a request that is expected (None: n); sm_scale: None for D ** -0.5;
    workspace_buf: uint8 device tensor of at least sd_kv_attend_workspace_bytes(D) bytes, or None
    for one that the call takes from the allocator and gives back (on its own stream, so that calls on
    several streams, threads or graphs do not meet).
    """
    cache = _cache_args(k_cache, v_cache, k_scale, v_scale)
    Hkv, D = k_cache.shape[2:]
    B, mb = block_table.shape
    if q.dim() != 3:
        raise SDError("q must be [tokens, Hq, D]")
    n, Hq = q.shape[:2]
    _int32(block_table, (B, mb), "block_table")
    _int32(ctx_lens, (B,), "ctx_lens")
    _int32(cu_q, (B + 1,), "cu_q")
    sq, so = _head_rows(q, Hq, D, "q"), _head_rows(out, Hq, D, "out")
    if out.shape[0] != n:
        raise SDError("out must have q's shape")
    if lse is not None and (lse.dtype != _t().float32 or lse.shape != (n, Hq)
                            or not lse.is_contiguous()):
        raise SDError("lse must be contiguous float32 [tokens, Hq]")
    raw, give = _raw_stream(k_cache, stream), None
    if workspace_buf is not None:
        ws, size = _ptr(workspace_buf), workspace_buf.numel()
    else:
        size = _attend_bytes.get(D)
        if size is None:
            size = _attend_bytes[D] = sd_kv_attend_workspace_bytes(D)
        ws, give = _take_scratch(k_cache, size, raw)
    try:
        rc = _quick().sd_kv_attend(B, n, max(1, n) if max_q is None else max_q, Hq, Hkv, D, _ptr(q),
                                   *sq, *cache, _ptr(block_table), mb, _ptr(ctx_lens), _ptr(cu_q),
                                   D ** -0.5 if sm_scale is None else sm_scale, int(bool(causal)),
                                   _ptr(out), *so, _ptr(lse), ws, size, _ptr(err), raw)
    finally:
        if give is not None:
            give(ws)
    _check(rc, "sd_kv_attend")


def sd_kv_weights(q, lse, k_cache, k_scale, block_table, ctx_lens, cu_q, weights, before=None,
                  live=None, max_q=None, sm_scale=None, causal=True, decay=1.0, err=None,
                  stream=None):
    """The attention weight that each cached token gets from a call's queries (see include/sd.h).

    q, block_table, ctx_lens, cu_q, max_q, sm_scale, causal: as for sd_kv_attend, and lse its [n, Hq]
    float32; live: [B] int32, how many of each request's query tokens count, or None for all; weights:
    [num_blocks, Hkv, block_size] float32; before: the same, what tokens had so far (it may be weights
    itself), or None; max_q: how many query tokens the longest request has, or None for n / B, rounded
    up: it only chooses the kernel (a batch with one prompt should say its length).
    """
    # (K alone is read: its checks serve for both)
    cache = _cache_args(k_cache, k_cache, k_scale, k_scale)
    nb, bs, Hkv, D = k_cache.shape
    B, mb = block_table.shape
    if q.dim() != 3:
        raise SDError("q must be [tokens, Hq, D]")
    n, Hq = q.shape[:2]
    _int32(block_table, (B, mb), "block_table")
    _int32(ctx_lens, (B,), "ctx_lens")
    _int32(cu_q, (B + 1,), "cu_q")
    if live is not None:
        _int32(live, (B,), "live")
    _float32(lse, (n, Hq), "lse")
    _float32(weights, (nb, Hkv, bs), "weights")
    if before is not None:
        _float32(before, (nb, Hkv, bs), "before")
    if max_q is None:
        max_q = max(1, -(-n // max(1, B)))
    rc = _quick().sd_kv_weights(B, n, max_q, Hq, Hkv, D, _ptr(q),
                                *_head_rows(q, Hq, D, "q"), _ptr(lse), cache[0], *cache[2:6], nb, bs,
                                _ptr(block_table), mb, _ptr(ctx_lens), _ptr(cu_q), _ptr(live),
                                D ** -0.5 if sm_scale is None else sm_scale, int(bool(causal)), decay,
                                _ptr(before), _ptr(weights), _ptr(err), _raw_stream(k_cache, stream))
    _check(rc, "sd_kv_weights")


def sd_kv_evict(k_cache, v_cache, k_scale, v_scale, weights, block_table, ctx_lens, kept, new_lens,
                to_table=None, sink=0, recent=0, err=None, stream=None):
    """Cut a cache to kept.shape[2] tokens a request, by their weights (see include/sd.h).

    weights: [num_blocks, Hkv, block_size] float32 (sd_kv_weights'); kept: [B, Hkv, budget] int32
    output, the positions that stay; new_lens: [B] int32 output; to_table: [B, blocks] int32, fresh
    pages for the tokens that stay, or None: they move to the front of the request's own.
    """
    cache = _cache_args(k_cache, v_cache, k_scale, v_scale)
    nb, bs, Hkv, D = k_cache.shape
    B, mb = block_table.shape
    _int32(block_table, (B, mb), "block_table")
    _int32(ctx_lens, (B,), "ctx_lens")
    _int32(new_lens, (B,), "new_lens")
    if kept.dim() != 3:
        raise SDError("kept must be [B, Hkv, budget]")
    budget = kept.shape[2]
    _int32(kept, (B, Hkv, budget), "kept")
    _float32(weights, (nb, Hkv, bs), "weights")
    to_blocks = 0
    if to_table is not None:
        to_blocks = to_table.shape[-1]
        _int32(to_table, (B, to_blocks), "to_table")
    rc = _quick().sd_kv_evict(B, Hkv, D, *cache, _ptr(weights), _ptr(block_table), mb,
                              _ptr(to_table), to_blocks, _ptr(ctx_lens), budget, sink, recent,
                              _ptr(kept), _ptr(new_lens), _ptr(err), _raw_stream(k_cache, stream))
    _check(rc, "sd_kv_evict")


_ROPE_PAIRS = {"halves": SD_ROPE_HALVES, "neighbours": SD_ROPE_NEIGHBOURS}
_ROPE_KINDS = {"plain": SD_ROPE_PLAIN, "linear": SD_ROPE_LINEAR, "ntk": SD_ROPE_NTK,
               "bands": SD_ROPE_BANDS, "yarn": SD_ROPE_YARN}


def sd_rope_table(rot, base=10000.0, kind="plain", factor=1.0, original_len=0, low=1.0, high=32.0,
                  device="cuda"):
    """(turns, scale) for sd_rope, made once for a model (see include/sd.h): turns [rot / 2] int64 on
    the device, the bits of fractions of 2^64; kind: "plain", "linear", "ntk", "bands" or "yarn"."""
    torch = _t()
    if kind not in _ROPE_KINDS:
        raise SDError(f"kind must be one of {sorted(_ROPE_KINDS)}")
    turns = torch.zeros(max(1, rot // 2), dtype=torch.int64)
    scale = ctypes.c_float()
    rc = _quick().sd_rope_table(rot, base, _ROPE_KINDS[kind], factor, original_len, low, high,
                                turns.data_ptr(), ctypes.byref(scale))
    _check(rc, "sd_rope_table")
    return turns.to(device), scale.value


def sd_rope(positions, turns, q=None, k=None, q_out=None, k_out=None, pairs="halves", scale=1.0,
            inverse=False, stream=None):
    """Rotary positions of queries and keys (see include/sd.h).

    positions: [n] int32; turns: [rot / 2] int64 (sd_rope_table's): the first rot values of a head
    turn; q, k: [n, heads, D] bfloat16 with contiguous heads (slices of one projection will do), either
    may be None; q_out, k_out: the same shapes, or None to turn them in place; pairs: "halves" or
    "neighbours"; inverse: turn back (a gradient; a turned key with 1 / scale).
    """
    if pairs not in _ROPE_PAIRS:
        raise SDError("pairs must be 'halves' or 'neighbours'")
    some = q if q is not None else k
    if some is None or some.dim() != 3:
        raise SDError("q and k must be [tokens, heads, D], one of them at least given")
    if turns.dtype != _t().int64 or turns.dim() != 1 or not turns.is_contiguous():
        raise SDError("turns must be contiguous int64 [rot / 2]")
    n, _, D = some.shape
    _int32(positions, (n,), "positions")
    args = []
    for x, y, what in ((q, q_out, "q"), (k, k_out, "k")):
        if x is None:
            if y is not None:
                raise SDError(f"{what}_out comes with {what}")
            args.append((0, None, 0, 0, None, 0, 0))
            continue
        if x.dim() != 3 or x.shape[0] != n:
            raise SDError("q and k must hold the same tokens")
        H = x.shape[1]
        y = x if y is None else y
        if y.shape != x.shape:
            raise SDError(f"{what}_out must have {what}'s shape")
        args.append((H, _ptr(x), *_head_rows(x, H, D, what), _ptr(y),
                     *_head_rows(y, H, D, what + "_out")))
    rc = _quick().sd_rope(n, args[0][0], args[1][0], D, 2 * turns.shape[0], _ROPE_PAIRS[pairs],
                          _ptr(positions), _ptr(turns), scale, int(bool(inverse)), *args[0][1:],
                          *args[1][1:], _raw_stream(some, stream))
    _check(rc, "sd_rope")


def _rows_args(rows, B, J, temperature, top_k, top_p, min_p):
    """The arguments that sd_truncate and sd_sample share."""
    torch = _t()
    if rows.dtype == torch.float32:
        dtype = SD_F32_PROBS
    elif rows.dtype == torch.bfloat16:
        dtype = SD_BF16_LOGITS
    else:
        raise SDError("rows must be float32 probabilities or bfloat16 logits")
    if rows.dim() != 2 or rows.shape[0] != B * J:
        raise SDError("rows must hold B*J rows")
    for t, what in ((temperature, "temperature"), (top_p, "top_p"), (min_p, "min_p")):
        if t is not None:
            _float32(t, (B,), what)
    if top_k is not None:
        _int32(top_k, (B,), "top_k")
    return (B, J, rows.shape[1], dtype, _ptr(rows), _row_stride(rows), _ptr(temperature), _ptr(top_k),
            _ptr(top_p), _ptr(min_p))


def sd_truncate(rows, probs, kept, temperature=None, top_k=None, top_p=None, min_p=None, err=None,
                stream=None):
    """Rows cut by top-k, top-p and min-p, as probability rows (see include/sd.h).

    rows: [B*J, V] float32 probabilities or bfloat16 logits; probs: [B*J, V] float32 output; kept:
    [B, J] int32 output, how many entries are kept (its shape says which rows are whose); temperature,
    top_p, min_p: [B] float32 or None; top_k: [B] int32 or None.
    """
    B, J = kept.shape
    args = _rows_args(rows, B, J, temperature, top_k, top_p, min_p)
    _int32(kept, (B, J), "kept")
    if probs.dtype != _t().float32 or probs.shape != rows.shape:
        raise SDError("probs must be float32 of rows' shape")
    rc = _quick().sd_truncate(*args, _ptr(probs), _row_stride(probs), _ptr(kept), _ptr(err),
                              _raw_stream(rows, stream))
    _check(rc, "sd_truncate")


def sd_sample(rows, u, tokens, prob=None, kept=None, temperature=None, top_k=None, top_p=None,
              min_p=None, err=None, stream=None):
    """One token drawn from each row, cut by top-k, top-p and min-p, by a given random number (see
    include/sd.h).

    rows: [B*J, V] float32 probabilities or bfloat16 logits; u: [B, J] float32 in [0, 1); tokens:
    [B, J] int32 output; prob: [B, J] float32 and kept: [B, J] int32 outputs or None; temperature,
    top_p, min_p: [B] float32 or None; top_k: [B] int32 or None.
    """
    B, J = tokens.shape
    args = _rows_args(rows, B, J, temperature, top_k, top_p, min_p)
    _int32(tokens, (B, J), "tokens")
    _float32(u, (B, J), "u")
    if prob is not None:
        _float32(prob, (B, J), "prob")
    if kept is not None:
        _int32(kept, (B, J), "kept")
    rc = _quick().sd_sample(*args, _ptr(u), _ptr(tokens), _ptr(prob), _ptr(kept), _ptr(err),
                            _raw_stream(rows, stream))
    _check(rc, "sd_sample")


def sd_token_logprobs(rows, tokens, logprob, entropy=None, rank=None, top_ids=None,
                      top_logprobs=None, temperature=None, err=None, stream=None):
    """Log probabilities of given tokens, with entropy, rank and alternatives (see include/sd.h).

    rows: [B*J, V] float32 probabilities or bfloat16 logits; tokens: [B, J] int32, -1 for none (a
    step's out_tokens); logprob, entropy: [B, J] float32; rank: [B, J] int32; top_ids,
    top_logprobs: [B, J, n_top] int32 and float32; temperature: [B] float32 or None. Every output
    but logprob may be None.
    """
    torch = _t()
    B, J = tokens.shape
    V = rows.shape[1]
    if rows.dtype == torch.float32:
        dtype = SD_F32_PROBS
    elif rows.dtype == torch.bfloat16:
        dtype = SD_BF16_LOGITS
    else:
        raise SDError("rows must be float32 probabilities or bfloat16 logits")
    if rows.shape[0] != B * J:
        raise SDError("rows must hold B*J rows")
    _int32(tokens, (B, J), "tokens")
    n_top = 0 if top_ids is None else top_ids.shape[-1]
    for t, dt, shape, what in ((logprob, torch.float32, (B, J), "logprob"),
                               (entropy, torch.float32, (B, J), "entropy"),
                               (rank, torch.int32, (B, J), "rank"),
                               (top_ids, torch.int32, (B, J, n_top), "top_ids"),
                               (top_logprobs, torch.float32, (B, J, n_top), "top_logprobs"),
                               (temperature, torch.float32, (B,), "temperature")):
        if t is not None and (t.dtype != dt or t.shape != shape or not t.is_contiguous()):
            raise SDError(f"{what} must be contiguous {dt} {list(shape)}")
    if n_top and top_logprobs is None:
        raise SDError("top_ids comes with top_logprobs")
    rc = _quick().sd_token_logprobs(B, J, V, dtype, _ptr(rows), _row_stride(rows), _ptr(tokens),
                                  _ptr(temperature), n_top, _ptr(logprob), _ptr(entropy),
                                  _ptr(rank), _ptr(top_ids), _ptr(top_logprobs), _ptr(err),
                                  _raw_stream(rows, stream))
    _check(rc, "sd_token_logprobs")
