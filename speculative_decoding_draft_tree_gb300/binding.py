"""Thin Python binding of the C-ABI in include/spec_verify.h (ctypes; argument marshalling only).

Every function here has the name of the C entry point it wraps, takes torch tensors that already
live on the GPU (device memory and streams are the only things torch provides), checks dtype /
device / contiguity, and calls the library on the current CUDA stream.  All computation happens
in the library's kernels; there is no CPU or PyTorch fallback: if libspecverify.so is missing or
fails to load, every call raises.
"""
import ctypes
import os

import torch

from . import build as _build

SPEC_OK, SPEC_ERR_INVALID_ARG, SPEC_ERR_UNSUPPORTED, SPEC_ERR_CUDA = 0, 1, 2, 3
SPEC_F32, SPEC_BF16, SPEC_E4M3 = 0, 1, 2
SPEC_DRAFT_LOGITS, SPEC_DRAFT_PROBS = 0, 1
SPEC_SIBLING_RESIDUAL, SPEC_SIBLING_INDEPENDENT, SPEC_SIBLING_MULTI_DRAFT = 0, 1, 2
SPEC_VERIFY_PATH_AUTO, SPEC_VERIFY_PATH_SPLIT, SPEC_VERIFY_PATH_WALK = 0, 1, 2
SPEC_MAX_TREE = 256
REQ_BITS = dict(BAD_PARENT=1, BAD_SIZE=2, BAD_TOKEN=4, BAD_DRAFT_ROW=8, BAD_DEPTH=16,
                BAD_BLOCK=32, TIMEOUT=64)
EXPORTS = ["spec_tree_build", "spec_tree_rope_kv_write", "spec_tree_build_rope_kv_write", "spec_tree_attention", "spec_attention_workspace_size",
           "spec_verify", "spec_verify_workspace_size", "spec_verify_noalloc", "spec_kv_compact",
           "spec_status_string", "spec_last_cuda_error", "spec_draft_init",
           "spec_draft_expand_select", "spec_draft_topk_append", "spec_echo_workspace_size",
           "spec_echo_select_pack", "spec_debug_draft_copy_stall", "spec_verify_compact",
           "spec_kernel_launches", "spec_kv8_append", "spec_tree_attention_kv8",
           "spec_attention_kv8_workspace_size", "spec_kv8_compact", "spec_kv_fork",
           "spec_tree_attention_window", "spec_attention_window_workspace_size",
           "spec_tree_attention_shared", "spec_attention_shared_workspace_size",
           "spec_beam_select", "spec_beam_select_workspace_size", "spec_beam_reorder",
           "spec_beam_reorder_workspace_size"]
SPEC_MAX_BEAMS = 16

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64


class SpecAttnParams(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", _i32), ("N", _i32), ("T_max", _i32),
                ("H_q", _i32), ("H_kv", _i32), ("head_dim", _i32), ("block_size", _i32),
                ("num_blocks", _i32), ("max_blocks_per_req", _i32), ("scale", ctypes.c_float),
                ("q", _vp), ("k_cache", _vp), ("v_cache", _vp), ("block_table", _vp),
                ("prefix_len", _vp), ("node_offset", _vp), ("anc_mask", _vp), ("o", _vp),
                ("lse", _vp), ("req_status", _vp)]


class SpecVerifyParams(ctypes.Structure):
    _fields_ = [("logits_dtype", ctypes.c_int), ("draft_kind", ctypes.c_int),
                ("sibling_rule", ctypes.c_int), ("B", _i32), ("N", _i32), ("R", _i32),
                ("V", _i32), ("target_ld", _i64), ("draft_ld", _i64), ("T_max", _i32),
                ("max_path", _i32), ("tau", ctypes.c_float), ("target", _vp), ("draft", _vp),
                ("draft_row", _vp), ("tokens", _vp), ("parent", _vp), ("node_offset", _vp),
                ("depth", _vp), ("is_internal", _vp), ("uniforms", _vp), ("req_status", _vp),
                ("out_tokens", _vp), ("out_len", _vp), ("path", _vp), ("n_acc", _vp),
                ("rejections", _vp), ("verify_path", _i32)]


class SpecCompactParams(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", _i32), ("H_kv", _i32), ("head_dim", _i32),
                ("block_size", _i32), ("num_blocks", _i32), ("max_blocks_per_req", _i32),
                ("num_layers", _i32), ("max_path", _i32), ("layer_stride", _i64),
                ("k_cache", _vp), ("v_cache", _vp), ("block_table", _vp), ("prefix_len", _vp),
                ("path", _vp), ("n_acc", _vp), ("req_status", _vp), ("new_kv_len", _vp),
                ("slot_map", _vp), ("blocks_in_use", _vp)]


class SpecRopeParams(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", _i32), ("N", _i32), ("H_q", _i32), ("H_kv", _i32),
                ("head_dim", _i32), ("rotary_dim", _i32), ("interleaved", _i32),
                ("block_size", _i32), ("num_blocks", _i32), ("max_blocks_per_req", _i32),
                ("base", ctypes.c_double), ("q_in", _vp), ("q_out", _vp), ("k_new", _vp),
                ("v_new", _vp), ("k_cache", _vp), ("v_cache", _vp), ("block_table", _vp),
                ("prefix_len", _vp), ("node_offset", _vp), ("pos_id", _vp), ("req_status", _vp)]


class SpecKv8AppendParams(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", _i32), ("N", _i32), ("H_kv", _i32),
                ("head_dim", _i32), ("block_size", _i32), ("num_blocks", _i32),
                ("max_blocks_per_req", _i32), ("k_ld", _i64), ("v_ld", _i64), ("k_new", _vp),
                ("v_new", _vp), ("k_cache", _vp), ("v_cache", _vp), ("k_scale", _vp),
                ("v_scale", _vp), ("block_table", _vp), ("start", _vp), ("row_offset", _vp),
                ("req_status", _vp)]


class SpecAttnKv8Params(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", _i32), ("N", _i32), ("T_max", _i32),
                ("H_q", _i32), ("H_kv", _i32), ("head_dim", _i32), ("block_size", _i32),
                ("num_blocks", _i32), ("max_blocks_per_req", _i32), ("scale", ctypes.c_float),
                ("q", _vp), ("k_cache", _vp), ("v_cache", _vp), ("k_scale", _vp),
                ("v_scale", _vp), ("block_table", _vp), ("prefix_len", _vp),
                ("node_offset", _vp), ("anc_mask", _vp), ("o", _vp), ("lse", _vp),
                ("req_status", _vp)]


class SpecKv8CompactParams(ctypes.Structure):
    _fields_ = [("B", _i32), ("H_kv", _i32), ("head_dim", _i32), ("block_size", _i32),
                ("num_blocks", _i32), ("max_blocks_per_req", _i32), ("num_layers", _i32),
                ("max_path", _i32), ("layer_stride", _i64), ("scale_layer_stride", _i64),
                ("k_cache", _vp), ("v_cache", _vp), ("k_scale", _vp), ("v_scale", _vp),
                ("block_table", _vp), ("prefix_len", _vp), ("path", _vp), ("n_acc", _vp),
                ("req_status", _vp), ("new_kv_len", _vp), ("slot_map", _vp),
                ("blocks_in_use", _vp)]


class SpecForkParams(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", _i32), ("F", _i32), ("H_kv", _i32),
                ("head_dim", _i32), ("block_size", _i32), ("num_blocks", _i32),
                ("max_blocks_per_req", _i32), ("num_layers", _i32), ("layer_stride", _i64),
                ("scale_layer_stride", _i64), ("k_cache", _vp), ("v_cache", _vp),
                ("k_scale", _vp), ("v_scale", _vp), ("block_table", _vp), ("kv_len", _vp),
                ("src", _vp), ("dst", _vp), ("new_block", _vp), ("fork_status", _vp)]


class SpecAttnWindowParams(ctypes.Structure):
    _fields_ = [("attn", SpecAttnParams), ("window", _i32), ("sinks", _i32)]


class SpecAttnSharedParams(ctypes.Structure):
    _fields_ = [("attn", SpecAttnParams), ("num_groups", _i32), ("group_offset", _vp),
                ("shared_len", _vp)]


class SpecBeamSelectParams(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", _i32), ("W", _i32), ("V", _i32), ("eos", _i32),
                ("ld", _i64), ("tau", ctypes.c_double), ("alpha", ctypes.c_double),
                ("logits", _vp), ("scores", _vp), ("lengths", _vp), ("finished", _vp),
                ("parent", _vp), ("token", _vp), ("out_score", _vp), ("out_length", _vp),
                ("out_finished", _vp)]


class SpecBeamReorderParams(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", _i32), ("W", _i32), ("H_kv", _i32),
                ("head_dim", _i32), ("block_size", _i32), ("num_blocks", _i32),
                ("max_blocks_per_req", _i32), ("num_layers", _i32), ("layer_stride", _i64),
                ("scale_layer_stride", _i64), ("k_cache", _vp), ("v_cache", _vp),
                ("k_scale", _vp), ("v_scale", _vp), ("block_table", _vp), ("kv_len", _vp),
                ("parent", _vp), ("beam_status", _vp)]


class SpecDraftPool(ctypes.Structure):
    _fields_ = [("B", _i32), ("cap", _i32), ("parent", _vp), ("token", _vp), ("depth", _vp),
                ("score", _vp), ("row", _vp), ("count", _vp)]


_LIB = None


def library_path():
    return _build.LIB_PATH


def load_library(build_if_missing=False):
    """Load libspecverify.so (building it first when asked); raises if it cannot be loaded."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if build_if_missing and not _build.up_to_date():
        _build.build_library()
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    st = ctypes.c_int
    lib.spec_tree_build.restype = st
    lib.spec_tree_build.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.spec_tree_rope_kv_write.restype = st
    lib.spec_tree_build_rope_kv_write.restype = st
    lib.spec_tree_build_rope_kv_write.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp,
                                                  _vp, _vp, ctypes.POINTER(SpecRopeParams), _vp]
    lib.spec_tree_rope_kv_write.argtypes = [ctypes.POINTER(SpecRopeParams), _vp]
    lib.spec_tree_attention.restype = st
    lib.spec_tree_attention.argtypes = [ctypes.POINTER(SpecAttnParams), _vp, ctypes.c_size_t, _vp]
    lib.spec_attention_workspace_size.restype = ctypes.c_size_t
    lib.spec_attention_workspace_size.argtypes = [ctypes.POINTER(SpecAttnParams)]
    lib.spec_verify.restype = st
    lib.spec_verify.argtypes = [ctypes.POINTER(SpecVerifyParams), _vp, ctypes.c_size_t, _vp]
    lib.spec_verify_noalloc.restype = st
    lib.spec_verify_noalloc.argtypes = [ctypes.POINTER(SpecVerifyParams), _vp]
    lib.spec_verify_workspace_size.restype = ctypes.c_size_t
    lib.spec_verify_workspace_size.argtypes = [ctypes.POINTER(SpecVerifyParams)]
    lib.spec_kv_compact.restype = st
    lib.spec_kv_compact.argtypes = [ctypes.POINTER(SpecCompactParams), _vp]
    lib.spec_draft_init.restype = st
    lib.spec_draft_init.argtypes = [ctypes.POINTER(SpecDraftPool), _vp, _vp]
    lib.spec_draft_expand_select.restype = st
    lib.spec_draft_expand_select.argtypes = [ctypes.POINTER(SpecDraftPool), _i32, _i32, _vp, _vp,
                                             _vp]
    lib.spec_draft_topk_append.restype = st
    lib.spec_draft_topk_append.argtypes = [ctypes.POINTER(SpecDraftPool), _i32, _i32, _vp,
                                           ctypes.c_int, _vp, _i64, _i32, ctypes.c_float, _i32,
                                           _vp, _vp]
    lib.spec_debug_draft_copy_stall.restype = st
    lib.spec_debug_draft_copy_stall.argtypes = [_i32]
    lib.spec_verify_compact.restype = st
    lib.spec_verify_compact.argtypes = [ctypes.POINTER(SpecVerifyParams),
                                        ctypes.POINTER(SpecCompactParams), _vp, ctypes.c_size_t,
                                        _vp]
    lib.spec_echo_workspace_size.restype = ctypes.c_size_t
    lib.spec_echo_workspace_size.argtypes = [_i32, _i32]
    lib.spec_echo_select_pack.restype = st
    lib.spec_echo_select_pack.argtypes = [ctypes.POINTER(SpecDraftPool), _i32, _vp, _vp, _vp,
                                          _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
    lib.spec_kv8_append.restype = st
    lib.spec_kv8_append.argtypes = [ctypes.POINTER(SpecKv8AppendParams), _vp]
    lib.spec_tree_attention_kv8.restype = st
    lib.spec_tree_attention_kv8.argtypes = [ctypes.POINTER(SpecAttnKv8Params), _vp,
                                            ctypes.c_size_t, _vp]
    lib.spec_attention_kv8_workspace_size.restype = ctypes.c_size_t
    lib.spec_attention_kv8_workspace_size.argtypes = [ctypes.POINTER(SpecAttnKv8Params)]
    lib.spec_kv8_compact.restype = st
    lib.spec_kv8_compact.argtypes = [ctypes.POINTER(SpecKv8CompactParams), _vp]
    lib.spec_kv_fork.restype = st
    lib.spec_kv_fork.argtypes = [ctypes.POINTER(SpecForkParams), _vp]
    for name, params in (("spec_tree_attention_window", SpecAttnWindowParams),
                         ("spec_tree_attention_shared", SpecAttnSharedParams),
                         ("spec_beam_select", SpecBeamSelectParams),
                         ("spec_beam_reorder", SpecBeamReorderParams)):
        getattr(lib, name).restype = st
        getattr(lib, name).argtypes = [ctypes.POINTER(params), _vp, ctypes.c_size_t, _vp]
        size = getattr(lib, name.replace("spec_tree_attention", "spec_attention") + "_workspace_size")
        size.restype, size.argtypes = ctypes.c_size_t, [ctypes.POINTER(params)]
    lib.spec_kernel_launches.restype = ctypes.c_uint64
    lib.spec_kernel_launches.argtypes = []
    lib.spec_status_string.restype = ctypes.c_char_p
    lib.spec_status_string.argtypes = [ctypes.c_int]
    lib.spec_last_cuda_error.restype = ctypes.c_int
    lib.spec_last_cuda_error.argtypes = []
    _LIB = lib
    return lib


class SpecError(RuntimeError):
    pass


def _check(code, what):
    if code != SPEC_OK:
        lib = load_library()
        msg = lib.spec_status_string(code).decode()
        if code == SPEC_ERR_CUDA:
            msg += f" (cudaError {lib.spec_last_cuda_error()})"
        raise SpecError(f"{what}: {msg}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, dtype, name, device=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    # the handle alone: building the stream object takes 3 us, as long as a small call
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise ValueError(f"unsupported dtype {t.dtype}")


# ----------------------------------------------------------------------------------------------
def spec_tree_build(parent, node_offset, prefix_len, T_max, depth, pos_id, anc_mask, is_internal,
                    req_status, stream=None):
    lib = load_library()
    i32 = torch.int32
    B = node_offset.numel() - 1
    N = parent.numel()
    for t, n in ((parent, "parent"), (node_offset, "node_offset"), (prefix_len, "prefix_len"),
                 (depth, "depth"), (pos_id, "pos_id"), (req_status, "req_status")):
        _need(t, i32, n)
    _need(anc_mask, torch.int32, "anc_mask")
    _need(is_internal, torch.uint8, "is_internal")
    code = lib.spec_tree_build(_ptr(parent), _ptr(node_offset), _ptr(prefix_len), B, N, T_max,
                               _ptr(depth), _ptr(pos_id), _ptr(anc_mask), _ptr(is_internal),
                               _ptr(req_status), _stream(stream))
    _check(code, "spec_tree_build")


def rope_params(q_in, q_out, k_new, v_new, k_cache, v_cache, block_table, prefix_len,
                node_offset, pos_id, req_status, base=10000.0, rotary_dim=None, interleaved=False):
    """k_cache / v_cache: one layer, [num_blocks, H_kv, block_size, head_dim]."""
    for t, n in ((q_in, "q_in"), (q_out, "q_out"), (k_new, "k_new"), (v_new, "v_new"),
                 (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, q_in.dtype, n)
    for t, n in ((block_table, "block_table"), (prefix_len, "prefix_len"),
                 (node_offset, "node_offset"), (pos_id, "pos_id"), (req_status, "req_status")):
        _need(t, torch.int32, n)
    p = SpecRopeParams()
    p.dtype = _dtype_code(q_in)
    p.B = node_offset.numel() - 1
    p.N, p.H_q, p.head_dim = q_in.shape
    p.H_kv = k_new.shape[1]
    if q_out.shape != q_in.shape or k_new.shape != (p.N, p.H_kv, p.head_dim) or v_new.shape != k_new.shape:
        raise ValueError("q_out must match q_in and v_new must match k_new [N, H_kv, head_dim]")
    p.rotary_dim = p.head_dim if rotary_dim is None else int(rotary_dim)
    p.interleaved = 1 if interleaved else 0
    p.num_blocks, _, p.block_size, _ = k_cache.shape
    p.max_blocks_per_req = block_table.shape[1]
    p.base = float(base)
    p.q_in, p.q_out, p.k_new, p.v_new = q_in.data_ptr(), q_out.data_ptr(), k_new.data_ptr(), v_new.data_ptr()
    p.k_cache, p.v_cache = k_cache.data_ptr(), v_cache.data_ptr()
    p.block_table, p.prefix_len = block_table.data_ptr(), prefix_len.data_ptr()
    p.node_offset, p.pos_id, p.req_status = node_offset.data_ptr(), pos_id.data_ptr(), req_status.data_ptr()
    return p


def spec_tree_build_rope_kv_write(parent, node_offset, prefix_len, T_max, depth, pos_id,
                                  anc_mask, is_internal, req_status, rope, stream=None):
    """spec_tree_build and spec_tree_rope_kv_write in one launch; `rope` from rope_params()
    over the same node_offset / prefix_len / pos_id / req_status."""
    lib = load_library()
    for t, n in ((parent, "parent"), (node_offset, "node_offset"), (prefix_len, "prefix_len"),
                 (depth, "depth"), (pos_id, "pos_id"), (req_status, "req_status"),
                 (anc_mask, "anc_mask")):
        _need(t, torch.int32, n)
    _need(is_internal, torch.uint8, "is_internal")
    code = lib.spec_tree_build_rope_kv_write(
        _ptr(parent), _ptr(node_offset), _ptr(prefix_len), node_offset.numel() - 1,
        parent.numel(), T_max, _ptr(depth), _ptr(pos_id), _ptr(anc_mask), _ptr(is_internal),
        _ptr(req_status), ctypes.byref(rope), _stream(stream))
    _check(code, "spec_tree_build_rope_kv_write")


def spec_tree_rope_kv_write(params, stream=None):
    code = load_library().spec_tree_rope_kv_write(ctypes.byref(params), _stream(stream))
    _check(code, "spec_tree_rope_kv_write")


def attention_params(q, k_cache, v_cache, block_table, prefix_len, node_offset, anc_mask, T_max,
                     o, lse, req_status, scale=0.0):
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (o, "o")):
        _need(t, None, n)
    for t, n in ((block_table, "block_table"), (prefix_len, "prefix_len"),
                 (node_offset, "node_offset"), (req_status, "req_status"),
                 (anc_mask, "anc_mask")):
        _need(t, torch.int32, n)
    if lse is not None:
        _need(lse, torch.float32, "lse")
    p = SpecAttnParams()
    p.dtype = _dtype_code(q)
    p.B = node_offset.numel() - 1
    p.N, p.H_q, p.head_dim = q.shape
    p.T_max = T_max
    p.num_blocks, p.H_kv, p.block_size = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
    p.max_blocks_per_req = block_table.shape[1]
    p.scale = scale
    p.q, p.k_cache, p.v_cache = q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
    p.block_table, p.prefix_len = block_table.data_ptr(), prefix_len.data_ptr()
    p.node_offset, p.anc_mask = node_offset.data_ptr(), anc_mask.data_ptr()
    p.o = o.data_ptr()
    p.lse = None if lse is None else lse.data_ptr()
    p.req_status = req_status.data_ptr()
    return p


def spec_attention_workspace_size(params):
    return int(load_library().spec_attention_workspace_size(ctypes.byref(params)))


def spec_tree_attention(params, workspace, stream=None):
    lib = load_library()
    wsz = 0 if workspace is None else workspace.numel() * workspace.element_size()
    code = lib.spec_tree_attention(ctypes.byref(params), _ptr(workspace), wsz, _stream(stream))
    _check(code, "spec_tree_attention")


def verify_params(target, draft, draft_kind, draft_row, tokens, parent, node_offset, depth,
                  is_internal, uniforms, tau, V, T_max, max_path, req_status, out_tokens,
                  out_len, path, n_acc, rejections=None, sibling_rule=SPEC_SIBLING_RESIDUAL,
                  verify_path=SPEC_VERIFY_PATH_AUTO):
    _need(target, None, "target")
    _need(draft, None, "draft")
    for t, n in ((draft_row, "draft_row"), (tokens, "tokens"), (parent, "parent"),
                 (node_offset, "node_offset"), (depth, "depth"), (req_status, "req_status"),
                 (out_tokens, "out_tokens"), (out_len, "out_len"), (path, "path"),
                 (n_acc, "n_acc")):
        _need(t, torch.int32, n)
    _need(is_internal, torch.uint8, "is_internal")
    _need(uniforms, torch.float32, "uniforms")
    p = SpecVerifyParams()
    p.logits_dtype = _dtype_code(target)
    p.draft_kind = draft_kind
    p.sibling_rule = sibling_rule
    p.B = node_offset.numel() - 1
    p.N = target.shape[0]
    p.R = draft.shape[0]
    p.V = V
    p.target_ld = target.shape[1]
    p.draft_ld = draft.shape[1]
    p.T_max, p.max_path, p.tau = T_max, max_path, float(tau)
    p.target, p.draft = target.data_ptr(), draft.data_ptr()
    p.draft_row, p.tokens, p.parent = draft_row.data_ptr(), tokens.data_ptr(), parent.data_ptr()
    p.node_offset, p.depth = node_offset.data_ptr(), depth.data_ptr()
    p.is_internal, p.uniforms = is_internal.data_ptr(), uniforms.data_ptr()
    p.req_status, p.out_tokens, p.out_len = req_status.data_ptr(), out_tokens.data_ptr(), out_len.data_ptr()
    p.path, p.n_acc = path.data_ptr(), n_acc.data_ptr()
    p.rejections = None if rejections is None else _need(rejections, torch.int32, "rejections").data_ptr()
    p.verify_path = int(verify_path)
    return p


def spec_verify_workspace_size(params):
    return int(load_library().spec_verify_workspace_size(ctypes.byref(params)))


def spec_verify(params, workspace, stream=None):
    lib = load_library()
    wsz = 0 if workspace is None else workspace.numel() * workspace.element_size()
    code = lib.spec_verify(ctypes.byref(params), _ptr(workspace), wsz, _stream(stream))
    _check(code, "spec_verify")


def spec_verify_noalloc(params, stream=None):
    """spec_verify without a caller workspace (see include/spec_verify.h): for callers that may
    not allocate device memory.  Calls whose kernels overlap on the GPU share one scratch array
    and race."""
    code = load_library().spec_verify_noalloc(ctypes.byref(params), _stream(stream))
    _check(code, "spec_verify_noalloc")


def spec_verify_compact(vparams, cparams, workspace, stream=None):
    """spec_verify then spec_kv_compact in one call (one kernel when the verification takes its
    one-launch form); cparams must name vparams' path, n_acc and req_status."""
    lib = load_library()
    wsz = 0 if workspace is None else workspace.numel() * workspace.element_size()
    code = lib.spec_verify_compact(ctypes.byref(vparams), ctypes.byref(cparams), _ptr(workspace),
                                   wsz, _stream(stream))
    _check(code, "spec_verify_compact")


def compact_params(k_cache, v_cache, block_table, prefix_len, path, n_acc, req_status,
                   new_kv_len, slot_map, blocks_in_use, max_path):
    """k_cache / v_cache: [L, num_blocks, H_kv, block_size, head_dim] (all layers)."""
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, None, n)
    for t, n in ((block_table, "block_table"), (prefix_len, "prefix_len"), (path, "path"),
                 (n_acc, "n_acc"), (req_status, "req_status"), (new_kv_len, "new_kv_len"),
                 (slot_map, "slot_map"), (blocks_in_use, "blocks_in_use")):
        _need(t, torch.int32, n)
    p = SpecCompactParams()
    p.dtype = _dtype_code(k_cache)
    L, nb, H_kv, bs, d = k_cache.shape
    p.B = block_table.shape[0]
    p.H_kv, p.head_dim, p.block_size, p.num_blocks = H_kv, d, bs, nb
    p.max_blocks_per_req = block_table.shape[1]
    p.num_layers, p.max_path = L, max_path
    p.layer_stride = nb * H_kv * bs * d
    p.k_cache, p.v_cache = k_cache.data_ptr(), v_cache.data_ptr()
    p.block_table, p.prefix_len = block_table.data_ptr(), prefix_len.data_ptr()
    p.path, p.n_acc, p.req_status = path.data_ptr(), n_acc.data_ptr(), req_status.data_ptr()
    p.new_kv_len, p.slot_map, p.blocks_in_use = new_kv_len.data_ptr(), slot_map.data_ptr(), blocks_in_use.data_ptr()
    return p


def spec_kv_compact(params, stream=None):
    code = load_library().spec_kv_compact(ctypes.byref(params), _stream(stream))
    _check(code, "spec_kv_compact")


# ----------------------------------------------------------------------------------------------
# The K/V cache in 8 bits: e4m3 codes (torch.float8_e4m3fn, or the same bytes as uint8) and one
# fp32 scale for each (block, KV head).
def _need_kv8(k_cache, v_cache, k_scale, v_scale, layers):
    """Checks an 8-bit cache ([L,] num_blocks, H_kv, block_size, head_dim; scales without the last
    two) and returns its shape."""
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, None, n)
        if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise ValueError(f"{n} must be torch.float8_e4m3fn or torch.uint8, got {t.dtype}")
        if t.dim() != 4 + layers or t.shape != k_cache.shape:
            raise ValueError(f"{n} must be [{'L, ' if layers else ''}num_blocks, H_kv, "
                             "block_size, head_dim], k_cache and v_cache alike")
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _need(t, torch.float32, n)
        if t.shape != k_cache.shape[:-2]:
            raise ValueError(f"{n} must be {tuple(k_cache.shape[:-2])}, got {tuple(t.shape)}")
    return tuple(k_cache.shape)


def _held(p, *tensors):
    """Keeps the tensors whose addresses `p` holds alive with it, and notes their device."""
    p._tensors = [t for t in tensors if t is not None]
    devices = {t.device for t in p._tensors}
    if len(devices) != 1:
        raise ValueError(f"all tensors must be on one device, got {sorted(map(str, devices))}")
    p._device = p._tensors[0].device.index
    return p


def _on_device(p):
    """The library launches on the current device: it has to be the tensors'."""
    if torch.cuda.current_device() != p._device:
        raise ValueError(f"the tensors are on cuda:{p._device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return ctypes.byref(p)


def _need_shape(t, shape, name, dtype=torch.int32):
    _need(t, dtype, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t


def kv8_append_params(k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_table, start,
                      row_offset, req_status):
    """k_new / v_new: [N, H_kv, head_dim] (fp32 or bf16; tokens may be strided, as slices of a
    fused projection are); k_cache / v_cache: one layer, [num_blocks, H_kv, block_size, head_dim];
    row row_offset[r] + i goes to slot start[r] + i of request r."""
    num_blocks, H_kv, bs, d = _need_kv8(k_cache, v_cache, k_scale, v_scale, 0)
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        if t is None or not t.is_cuda:
            raise ValueError(f"{n} must be a CUDA tensor")
        if t.dtype != k_new.dtype:
            raise ValueError(f"{n} must be {k_new.dtype}, got {t.dtype}")
        if t.dim() != 3 or tuple(t.shape) != (k_new.shape[0], H_kv, d):
            raise ValueError(f"{n} must be [N, {H_kv}, {d}], got {tuple(t.shape)}")
        if t.shape[0] > 0 and (t.stride(2) != 1 or (H_kv > 1 and t.stride(1) != d)):
            raise ValueError(f"{n}: the rows of a token must be contiguous")
    B = block_table.shape[0]
    _need(block_table, torch.int32, "block_table")
    _need_shape(start, (B,), "start")
    _need_shape(row_offset, (B + 1,), "row_offset")
    _need_shape(req_status, (B,), "req_status")
    p = SpecKv8AppendParams()
    p.dtype = _dtype_code(k_new)
    p.B, p.N, p.H_kv, p.head_dim = B, k_new.shape[0], H_kv, d
    p.block_size, p.num_blocks, p.max_blocks_per_req = bs, num_blocks, block_table.shape[1]
    p.k_ld = k_new.stride(0) if p.N > 1 else H_kv * d
    p.v_ld = v_new.stride(0) if p.N > 1 else H_kv * d
    p.k_new, p.v_new = k_new.data_ptr(), v_new.data_ptr()
    p.k_cache, p.v_cache = k_cache.data_ptr(), v_cache.data_ptr()
    p.k_scale, p.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
    p.block_table, p.start = block_table.data_ptr(), start.data_ptr()
    p.row_offset, p.req_status = row_offset.data_ptr(), req_status.data_ptr()
    return _held(p, k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_table, start,
                 row_offset, req_status)


def spec_kv8_append(params, stream=None):
    """Quantise new K/V rows into the 8-bit cache (params from kv8_append_params)."""
    code = load_library().spec_kv8_append(_on_device(params), _stream(stream))
    _check(code, "spec_kv8_append")


def attention_kv8_params(q, k_cache, v_cache, k_scale, v_scale, block_table, prefix_len,
                         node_offset, anc_mask, T_max, o, lse, req_status, scale=0.0):
    """attention_params over one layer of an 8-bit cache; lse may be None."""
    num_blocks, H_kv, bs, d = _need_kv8(k_cache, v_cache, k_scale, v_scale, 0)
    _need(q, None, "q")
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError(f"q must be [N, H_q, {d}], got {tuple(q.shape)}")
    N, H_q = q.shape[0], q.shape[1]
    _need_shape(o, q.shape, "o", q.dtype)
    if lse is not None:
        _need_shape(lse, (N, H_q), "lse", torch.float32)
    B = block_table.shape[0]
    _need(block_table, torch.int32, "block_table")
    _need_shape(prefix_len, (B,), "prefix_len")
    _need_shape(node_offset, (B + 1,), "node_offset")
    _need_shape(anc_mask, (N, (int(T_max) + 31) // 32), "anc_mask")
    _need_shape(req_status, (B,), "req_status")
    p = SpecAttnKv8Params()
    p.dtype = _dtype_code(q)
    p.B, p.N, p.T_max, p.H_q, p.H_kv, p.head_dim = B, N, int(T_max), H_q, H_kv, d
    p.block_size, p.num_blocks, p.max_blocks_per_req = bs, num_blocks, block_table.shape[1]
    p.scale = scale
    p.q, p.k_cache, p.v_cache = q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
    p.k_scale, p.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
    p.block_table, p.prefix_len = block_table.data_ptr(), prefix_len.data_ptr()
    p.node_offset, p.anc_mask = node_offset.data_ptr(), anc_mask.data_ptr()
    p.o, p.lse = o.data_ptr(), None if lse is None else lse.data_ptr()
    p.req_status = req_status.data_ptr()
    return _held(p, q, k_cache, v_cache, k_scale, v_scale, block_table, prefix_len, node_offset,
                 anc_mask, o, lse, req_status)


def spec_attention_kv8_workspace_size(params):
    return int(load_library().spec_attention_kv8_workspace_size(ctypes.byref(params)))


def spec_tree_attention_kv8(params, workspace, stream=None):
    """Tree attention over the 8-bit cache; calls that may overlap need a workspace each."""
    if workspace is not None:
        _need(workspace, None, "workspace")
        if workspace.device.index != params._device:
            raise ValueError(f"workspace must be on cuda:{params._device}")
    wsz = 0 if workspace is None else workspace.numel() * workspace.element_size()
    code = load_library().spec_tree_attention_kv8(_on_device(params), _ptr(workspace), wsz,
                                                  _stream(stream))
    _check(code, "spec_tree_attention_kv8")


def kv8_compact_params(k_cache, v_cache, k_scale, v_scale, block_table, prefix_len, path, n_acc,
                       req_status, new_kv_len, slot_map, blocks_in_use, max_path):
    """compact_params for an 8-bit cache: [L, num_blocks, H_kv, block_size, head_dim], scales
    [L, num_blocks, H_kv]."""
    L, nb, H_kv, bs, d = _need_kv8(k_cache, v_cache, k_scale, v_scale, 1)
    B = block_table.shape[0]
    _need(block_table, torch.int32, "block_table")
    for t, n in ((prefix_len, "prefix_len"), (n_acc, "n_acc"), (req_status, "req_status"),
                 (new_kv_len, "new_kv_len"), (blocks_in_use, "blocks_in_use")):
        _need_shape(t, (B,), n)
    _need_shape(path, (B, max_path), "path")
    _need_shape(slot_map, (B, max_path, 2), "slot_map")
    p = SpecKv8CompactParams()
    p.B, p.H_kv, p.head_dim, p.block_size, p.num_blocks = B, H_kv, d, bs, nb
    p.max_blocks_per_req, p.num_layers, p.max_path = block_table.shape[1], L, max_path
    p.layer_stride, p.scale_layer_stride = nb * H_kv * bs * d, nb * H_kv
    p.k_cache, p.v_cache = k_cache.data_ptr(), v_cache.data_ptr()
    p.k_scale, p.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
    p.block_table, p.prefix_len = block_table.data_ptr(), prefix_len.data_ptr()
    p.path, p.n_acc, p.req_status = path.data_ptr(), n_acc.data_ptr(), req_status.data_ptr()
    p.new_kv_len, p.slot_map = new_kv_len.data_ptr(), slot_map.data_ptr()
    p.blocks_in_use = blocks_in_use.data_ptr()
    return _held(p, k_cache, v_cache, k_scale, v_scale, block_table, prefix_len, path, n_acc,
                 req_status, new_kv_len, slot_map, blocks_in_use)


def spec_kv8_compact(params, stream=None):
    """Commit the accepted path in the 8-bit cache, every layer (params from kv8_compact_params)."""
    code = load_library().spec_kv8_compact(_on_device(params), _stream(stream))
    _check(code, "spec_kv8_compact")


def kv_fork_params(k_cache, v_cache, block_table, kv_len, src, dst, new_block, fork_status,
                   k_scale=None, v_scale=None):
    """k_cache / v_cache: [L, num_blocks, H_kv, block_size, head_dim], fp32, bf16 or 8-bit (then
    with k_scale / v_scale [L, num_blocks, H_kv]); block_table [B, max_blocks], kv_len [B] (both
    updated); src, dst, new_block, fork_status [F]."""
    if k_scale is not None or v_scale is not None:
        L, nb, H_kv, bs, d = _need_kv8(k_cache, v_cache, k_scale, v_scale, 1)
        code = SPEC_E4M3
    else:
        _need(k_cache, None, "k_cache")
        code = _dtype_code(k_cache)
        if k_cache.dim() != 5:
            raise ValueError("k_cache must be [L, num_blocks, H_kv, block_size, head_dim]")
        _need_shape(v_cache, k_cache.shape, "v_cache", k_cache.dtype)
        L, nb, H_kv, bs, d = k_cache.shape
    _need(block_table, torch.int32, "block_table")
    _need_shape(kv_len, (block_table.shape[0],), "kv_len")
    F = src.numel()
    for t, n in ((src, "src"), (dst, "dst"), (new_block, "new_block"),
                 (fork_status, "fork_status")):
        _need_shape(t, (F,), n)
    p = SpecForkParams()
    p.dtype, p.B, p.F = code, block_table.shape[0], F
    p.H_kv, p.head_dim, p.block_size, p.num_blocks = H_kv, d, bs, nb
    p.max_blocks_per_req, p.num_layers = block_table.shape[1], L
    p.layer_stride, p.scale_layer_stride = nb * H_kv * bs * d, nb * H_kv
    p.k_cache, p.v_cache = k_cache.data_ptr(), v_cache.data_ptr()
    p.k_scale = None if k_scale is None else k_scale.data_ptr()
    p.v_scale = None if v_scale is None else v_scale.data_ptr()
    p.block_table, p.kv_len = block_table.data_ptr(), kv_len.data_ptr()
    p.src, p.dst, p.new_block = src.data_ptr(), dst.data_ptr(), new_block.data_ptr()
    p.fork_status = fork_status.data_ptr()
    return _held(p, k_cache, v_cache, block_table, kv_len, src, dst, new_block, fork_status,
                 k_scale, v_scale)


def spec_kv_fork(params, stream=None):
    """Child sequences of cached ones: shared full pages, the partial page copied."""
    code = load_library().spec_kv_fork(_on_device(params), _stream(stream))
    _check(code, "spec_kv_fork")


# ----------------------------------------------------------------------------------------------
# Attention over a window of the cache, or over a prefix that requests have in common; beam search.
def _paged_attention(q, k_cache, v_cache, block_table, prefix_len, node_offset, anc_mask, T_max, o,
                     lse, req_status, scale):
    """attention_params with every shape checked: one layer's caches [num_blocks, H_kv, block_size,
    head_dim], q and o [N, H_q, head_dim]."""
    _need(q, None, "q")
    if q.dim() != 3:
        raise ValueError(f"q must be [N, H_q, head_dim], got {tuple(q.shape)}")
    N, H_q, d = q.shape
    _need(k_cache, q.dtype, "k_cache")
    if k_cache.dim() != 4 or k_cache.shape[3] != d:
        raise ValueError(f"k_cache must be [num_blocks, H_kv, block_size, {d}], got "
                         f"{tuple(k_cache.shape)}")
    _need_shape(v_cache, k_cache.shape, "v_cache", q.dtype)
    _need_shape(o, q.shape, "o", q.dtype)
    if lse is not None:
        _need_shape(lse, (N, H_q), "lse", torch.float32)
    _need(block_table, torch.int32, "block_table")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks]")
    B = block_table.shape[0]
    _need_shape(prefix_len, (B,), "prefix_len")
    _need_shape(node_offset, (B + 1,), "node_offset")
    _need_shape(anc_mask, (N, (int(T_max) + 31) // 32), "anc_mask")
    _need_shape(req_status, (B,), "req_status")
    return attention_params(q, k_cache, v_cache, block_table, prefix_len, node_offset, anc_mask,
                            int(T_max), o, lse, req_status, scale)


def _call(name, params, workspace, stream):
    if workspace is not None:
        _need(workspace, None, "workspace")
        if workspace.device.index != params._device:
            raise ValueError(f"workspace must be on cuda:{params._device}")
    wsz = 0 if workspace is None else workspace.numel() * workspace.element_size()
    code = getattr(load_library(), name)(_on_device(params), _ptr(workspace), wsz, _stream(stream))
    _check(code, name)


def attention_window_params(q, k_cache, v_cache, block_table, prefix_len, node_offset, anc_mask,
                            T_max, window, sinks, o, lse, req_status, scale=0.0):
    """attention_params with a sliding window: a node sees the last `window` positions up to its own
    and the first `sinks`.  Table entries of pages that no node sees may hold anything (-1)."""
    p = SpecAttnWindowParams()
    p.attn = _paged_attention(q, k_cache, v_cache, block_table, prefix_len, node_offset, anc_mask,
                              T_max, o, lse, req_status, scale)
    p.window, p.sinks = int(window), int(sinks)
    return _held(p, q, k_cache, v_cache, block_table, prefix_len, node_offset, anc_mask, o, lse,
                 req_status)


def spec_attention_window_workspace_size(params):
    return int(load_library().spec_attention_window_workspace_size(ctypes.byref(params)))


def spec_tree_attention_window(params, workspace, stream=None):
    """Tree attention with a sliding window and sinks; calls that may overlap need a workspace each."""
    _call("spec_tree_attention_window", params, workspace, stream)


def attention_shared_params(q, k_cache, v_cache, block_table, prefix_len, node_offset, anc_mask,
                            T_max, group_offset, shared_len, o, lse, req_status, scale=0.0):
    """attention_params for groups of consecutive requests (group_offset [groups + 1]) that have their
    first shared_len [groups] slots in common; those are read once a group, by its first request's
    table row."""
    p = SpecAttnSharedParams()
    p.attn = _paged_attention(q, k_cache, v_cache, block_table, prefix_len, node_offset, anc_mask,
                              T_max, o, lse, req_status, scale)
    _need(shared_len, torch.int32, "shared_len")
    _need_shape(group_offset, (shared_len.numel() + 1,), "group_offset")
    p.num_groups = shared_len.numel()
    p.group_offset, p.shared_len = group_offset.data_ptr(), shared_len.data_ptr()
    return _held(p, q, k_cache, v_cache, block_table, prefix_len, node_offset, anc_mask, o, lse,
                 req_status, group_offset, shared_len)


def spec_attention_shared_workspace_size(params):
    return int(load_library().spec_attention_shared_workspace_size(ctypes.byref(params)))


def spec_tree_attention_shared(params, workspace, stream=None):
    """Tree attention under shared prefixes; calls that may overlap need a workspace each."""
    _call("spec_tree_attention_shared", params, workspace, stream)


def beam_select_params(logits, V, tau, scores, lengths, finished, eos, alpha, parent, token,
                       out_score, out_length, out_finished):
    """logits [B * W, ld] (fp32 or bf16, ld >= V); scores fp32, lengths, finished and the outputs
    int32 (out_score fp32), all [B, W].  The outputs of score, length and finished may be the inputs'
    own tensors."""
    _need(scores, torch.float32, "scores")
    if scores.dim() != 2:
        raise ValueError("scores must be [B, W]")
    B, W = scores.shape
    _need(logits, None, "logits")
    if logits.dim() != 2 or logits.shape[0] != B * W:
        raise ValueError(f"logits must be [{B * W}, ld], got {tuple(logits.shape)}")
    for t, n in ((lengths, "lengths"), (finished, "finished"), (parent, "parent"),
                 (token, "token"), (out_length, "out_length"), (out_finished, "out_finished")):
        _need_shape(t, (B, W), n)
    _need_shape(out_score, (B, W), "out_score", torch.float32)
    p = SpecBeamSelectParams()
    p.dtype = _dtype_code(logits)
    p.B, p.W, p.V, p.eos, p.ld = B, W, int(V), int(eos), logits.shape[1]
    p.tau, p.alpha = float(tau), float(alpha)
    p.logits, p.scores, p.lengths = logits.data_ptr(), scores.data_ptr(), lengths.data_ptr()
    p.finished, p.parent, p.token = finished.data_ptr(), parent.data_ptr(), token.data_ptr()
    p.out_score, p.out_length = out_score.data_ptr(), out_length.data_ptr()
    p.out_finished = out_finished.data_ptr()
    return _held(p, logits, scores, lengths, finished, parent, token, out_score, out_length,
                 out_finished)


def spec_beam_select_workspace_size(params):
    return int(load_library().spec_beam_select_workspace_size(ctypes.byref(params)))


def spec_beam_select(params, workspace, stream=None):
    """The best W continuations of each request's W beams (params from beam_select_params)."""
    _call("spec_beam_select", params, workspace, stream)


def beam_reorder_params(k_cache, v_cache, block_table, kv_len, parent, beam_status, k_scale=None,
                        v_scale=None):
    """k_cache / v_cache: [L, num_blocks, H_kv, block_size, head_dim], fp32, bf16 or 8-bit (then with
    k_scale / v_scale [L, num_blocks, H_kv]); block_table [B * W, max_blocks] (updated), kv_len,
    beam_status [B], parent [B, W]."""
    if k_scale is not None or v_scale is not None:
        L, nb, H_kv, bs, d = _need_kv8(k_cache, v_cache, k_scale, v_scale, 1)
        code = SPEC_E4M3
    else:
        _need(k_cache, None, "k_cache")
        code = _dtype_code(k_cache)
        if k_cache.dim() != 5:
            raise ValueError("k_cache must be [L, num_blocks, H_kv, block_size, head_dim]")
        _need_shape(v_cache, k_cache.shape, "v_cache", k_cache.dtype)
        L, nb, H_kv, bs, d = k_cache.shape
    _need(parent, torch.int32, "parent")
    if parent.dim() != 2:
        raise ValueError("parent must be [B, W]")
    B, W = parent.shape
    _need(block_table, torch.int32, "block_table")
    if block_table.dim() != 2 or block_table.shape[0] != B * W:
        raise ValueError(f"block_table must be [{B * W}, max_blocks], got "
                         f"{tuple(block_table.shape)}")
    _need_shape(kv_len, (B,), "kv_len")
    _need_shape(beam_status, (B,), "beam_status")
    p = SpecBeamReorderParams()
    p.dtype, p.B, p.W = code, B, W
    p.H_kv, p.head_dim, p.block_size, p.num_blocks = H_kv, d, bs, nb
    p.max_blocks_per_req, p.num_layers = block_table.shape[1], L
    p.layer_stride, p.scale_layer_stride = nb * H_kv * bs * d, nb * H_kv
    p.k_cache, p.v_cache = k_cache.data_ptr(), v_cache.data_ptr()
    p.k_scale = None if k_scale is None else k_scale.data_ptr()
    p.v_scale = None if v_scale is None else v_scale.data_ptr()
    p.block_table, p.kv_len = block_table.data_ptr(), kv_len.data_ptr()
    p.parent, p.beam_status = parent.data_ptr(), beam_status.data_ptr()
    return _held(p, k_cache, v_cache, block_table, kv_len, parent, beam_status, k_scale, v_scale)


def spec_beam_reorder_workspace_size(params):
    return int(load_library().spec_beam_reorder_workspace_size(ctypes.byref(params)))


def spec_beam_reorder(params, workspace, stream=None):
    """The beams' cache follows the selection, in place (params from beam_reorder_params)."""
    _call("spec_beam_reorder", params, workspace, stream)


# ----------------------------------------------------------------------------------------------
def draft_pool(parent, token, depth, score, row, count):
    """The candidate pool ([B, cap] int32 / fp32 arrays and count [B])."""
    for t, n in ((parent, "parent"), (token, "token"), (depth, "depth"), (row, "row"),
                 (count, "count")):
        _need(t, torch.int32, n)
    _need(score, torch.float32, "score")
    p = SpecDraftPool()
    p.B, p.cap = parent.shape
    p.parent, p.token, p.depth = parent.data_ptr(), token.data_ptr(), depth.data_ptr()
    p.score, p.row, p.count = score.data_ptr(), row.data_ptr(), count.data_ptr()
    return p


def spec_draft_init(pool, root_tokens, stream=None):
    _need(root_tokens, torch.int32, "root_tokens")
    _check(load_library().spec_draft_init(ctypes.byref(pool), _ptr(root_tokens), _stream(stream)),
           "spec_draft_init")


def spec_draft_expand_select(pool, level, K, expand, req_status=None, stream=None):
    _need(expand, torch.int32, "expand")
    code = load_library().spec_draft_expand_select(ctypes.byref(pool), level, K, _ptr(expand),
                                                   _ptr(req_status), _stream(stream))
    _check(code, "spec_draft_expand_select")


def spec_draft_topk_append(pool, level, K, expand, rows, V, tau, row_base, req_status=None,
                           stream=None):
    _need(expand, torch.int32, "expand")
    _need(rows, None, "rows")
    code = load_library().spec_draft_topk_append(ctypes.byref(pool), level, K, _ptr(expand),
                                                 _dtype_code(rows), _ptr(rows), rows.shape[1], V,
                                                 float(tau), row_base, _ptr(req_status),
                                                 _stream(stream))
    _check(code, "spec_draft_topk_append")


def spec_echo_workspace_size(B, cap):
    return int(load_library().spec_echo_workspace_size(B, cap))


def spec_echo_select_pack(pool, K_max, node_offset, parent, tokens, depth, draft_row, source,
                          workspace, stream=None):
    for t, n in ((node_offset, "node_offset"), (parent, "parent"), (tokens, "tokens"),
                 (depth, "depth"), (draft_row, "draft_row")):
        _need(t, torch.int32, n)
    wsz = workspace.numel() * workspace.element_size()
    code = load_library().spec_echo_select_pack(ctypes.byref(pool), K_max, _ptr(node_offset),
                                                _ptr(parent), _ptr(tokens), _ptr(depth),
                                                _ptr(draft_row), _ptr(source), _ptr(workspace),
                                                wsz, _stream(stream))
    _check(code, "spec_echo_select_pack")


def spec_debug_draft_copy_stall(chunk):
    """Testing only: make the next top-K launches lose one chunk's copy (-1: off)."""
    _check(load_library().spec_debug_draft_copy_stall(int(chunk)), "spec_debug_draft_copy_stall")


def spec_kernel_launches():
    """Kernels the library has enqueued in this process so far (a launch captured into a CUDA
    graph counts once, when captured; graph replays do not count)."""
    return int(load_library().spec_kernel_launches())
