"""Host side of windowed and shared-prefix attention and of beam search: struct layouts and refusals, before any
CUDA call."""
import ctypes
import subprocess

import pytest
import torch

from speculative_decoding_draft_tree_gb300 import binding as B
from speculative_decoding_draft_tree_gb300 import build

FAKE = 0x100000   # 256-byte aligned, never dereferenced: validation fails first
INV, UNS = B.SPEC_ERR_INVALID_ARG, B.SPEC_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return B.load_library()


def test_struct_layouts_match_header(tmp_path):
    structs = {"spec_attn_window_params": B.SpecAttnWindowParams, "spec_attn_shared_params": B.SpecAttnSharedParams,
               "spec_beam_select_params": B.SpecBeamSelectParams, "spec_beam_reorder_params": B.SpecBeamReorderParams}
    lines, want = ["#include <stdio.h>", "#include <stddef.h>", '#include "spec_verify.h"', "int main(void) {"], []
    for cname, py in structs.items():
        lines.append(f'  printf("%zu\\n", sizeof({cname}));')
        want.append(ctypes.sizeof(py))
        for f, _ in py._fields_:
            lines.append(f'  printf("%zu\\n", offsetof({cname}, {f}));')
            want.append(getattr(py, f).offset)
    lines += ['  printf("%d\\n", SPEC_MAX_BEAMS);', "  return 0;", "}"]
    want.append(B.SPEC_MAX_BEAMS)
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-I", build.INCLUDE, str(src), "-o", str(exe)], check=True)
    assert [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()] == want


def _fill(p, **kw):
    for f, t in p._fields_:
        if t is ctypes.c_void_p:
            setattr(p, f, FAKE)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


ATTN = dict(dtype=1, B=2, N=4, T_max=2, H_q=4, H_kv=2, head_dim=128, block_size=16, num_blocks=8, max_blocks_per_req=4, scale=0.0)
BAD_ATTN = [(dict(dtype=2), INV), (dict(B=0), INV), (dict(N=-1), INV), (dict(T_max=0), INV), (dict(T_max=257), INV), (dict(H_q=3), INV),
            (dict(H_q=0), INV), (dict(H_kv=0), INV), (dict(head_dim=0), INV), (dict(head_dim=12), INV), (dict(head_dim=264), UNS),
            (dict(block_size=0), INV), (dict(num_blocks=0), INV), (dict(num_blocks=1 << 30), UNS), (dict(max_blocks_per_req=0), INV),
            (dict(q=None), INV), (dict(o=FAKE + 4), INV), (dict(k_cache=None), INV), (dict(v_cache=FAKE + 8), INV),
            (dict(anc_mask=None), INV), (dict(prefix_len=None), INV), (dict(node_offset=None), INV), (dict(block_table=None), INV),
            (dict(req_status=None), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV)]


@pytest.mark.parametrize("change,code", BAD_ATTN)
def test_attention_refusals(lib, change, code):
    w, s = B.SpecAttnWindowParams(), B.SpecAttnSharedParams()
    _fill(w.attn, **{**ATTN, **change})
    _fill(s.attn, **{**ATTN, **change})
    w.window, w.sinks = 4, 1
    s.num_groups, s.group_offset, s.shared_len = 1, FAKE, FAKE
    assert lib.spec_tree_attention_window(ctypes.byref(w), FAKE, 1 << 40, None) == code
    assert lib.spec_tree_attention_shared(ctypes.byref(s), FAKE, 1 << 40, None) == code
    assert lib.spec_attention_window_workspace_size(ctypes.byref(w)) == lib.spec_attention_shared_workspace_size(ctypes.byref(s)) == 0


def test_window_and_group_refusals(lib):
    for window, sinks in ((0, 0), (-1, 0), (4, -1)):
        w = B.SpecAttnWindowParams()
        _fill(w.attn, **ATTN)
        w.window, w.sinks = window, sinks
        assert lib.spec_tree_attention_window(ctypes.byref(w), FAKE, 1 << 40, None) == INV
        assert lib.spec_attention_window_workspace_size(ctypes.byref(w)) == 0
    for groups, off, ln in ((0, FAKE, FAKE), (3, FAKE, FAKE), (-1, FAKE, FAKE), (1, None, FAKE), (1, FAKE, None)):
        s = B.SpecAttnSharedParams()
        _fill(s.attn, **ATTN)
        s.num_groups, s.group_offset, s.shared_len = groups, off, ln
        assert lib.spec_tree_attention_shared(ctypes.byref(s), FAKE, 1 << 40, None) == INV
        assert lib.spec_attention_shared_workspace_size(ctypes.byref(s)) == 0


SELECT = dict(dtype=1, B=2, W=3, V=50, eos=2, ld=56, tau=1.0, alpha=0.0)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), INV), (dict(B=0), INV), (dict(W=0), INV), (dict(W=17), UNS), (dict(V=0), INV), (dict(ld=49), INV), (dict(ld=52), INV),
    (dict(tau=0.0), INV), (dict(tau=-1.0), INV), (dict(tau=float("nan")), INV), (dict(tau=float("inf")), INV), (dict(tau=1e-39), INV),
    (dict(tau=1e39), INV), (dict(alpha=-0.1), INV), (dict(alpha=float("nan")), INV), (dict(alpha=float("inf")), INV),
    (dict(logits=None), INV), (dict(logits=FAKE + 8), INV), (dict(scores=None), INV), (dict(lengths=None), INV),
    (dict(finished=None), INV), (dict(parent=None), INV), (dict(token=None), INV), (dict(out_score=None), INV),
    (dict(out_length=None), INV), (dict(out_finished=None), INV), (dict(B=30000), UNS)])
def test_select_refusals(lib, change, code):
    p = _fill(B.SpecBeamSelectParams(), **{**SELECT, **change})
    assert lib.spec_beam_select(ctypes.byref(p), FAKE, 1 << 40, None) == code
    assert lib.spec_beam_select_workspace_size(ctypes.byref(p)) == 0


REORDER = dict(dtype=1, B=2, W=3, H_kv=2, head_dim=128, block_size=16, num_blocks=8, max_blocks_per_req=4, num_layers=2, layer_stride=4096, scale_layer_stride=0)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), INV), (dict(B=0), INV), (dict(W=0), INV), (dict(W=17), UNS), (dict(H_kv=0), INV), (dict(head_dim=4), INV),
    (dict(block_size=0), INV), (dict(num_blocks=0), INV), (dict(max_blocks_per_req=0), INV), (dict(num_layers=0), INV),
    (dict(num_layers=65536), UNS), (dict(layer_stride=-16), INV), (dict(layer_stride=12), INV), (dict(scale_layer_stride=-1), INV),
    (dict(k_cache=None), INV), (dict(v_cache=FAKE + 4), INV), (dict(block_table=None), INV), (dict(kv_len=None), INV),
    (dict(parent=None), INV), (dict(beam_status=None), INV), (dict(dtype=2, k_scale=None), INV), (dict(block_size=1 << 30), UNS),
    (dict(B=1 << 30), UNS)])
def test_reorder_refusals(lib, change, code):
    p = _fill(B.SpecBeamReorderParams(), **{**REORDER, **change})
    assert lib.spec_beam_reorder(ctypes.byref(p), FAKE, 1 << 40, None) == code
    assert lib.spec_beam_reorder_workspace_size(ctypes.byref(p)) == 0


def test_null_and_empty_calls(lib):
    for name in ("spec_tree_attention_window", "spec_tree_attention_shared", "spec_beam_select", "spec_beam_reorder"):
        assert getattr(lib, name)(None, None, 0, None) == INV
    w, s = B.SpecAttnWindowParams(), B.SpecAttnSharedParams()
    for p in (w, s):
        _fill(p.attn, **{**ATTN, **dict(N=0, q=None, o=None, k_cache=None, v_cache=None, anc_mask=None)})
    w.window, s.num_groups, s.group_offset, s.shared_len = 1, 2, FAKE, FAKE
    assert lib.spec_tree_attention_window(ctypes.byref(w), None, 0, None) == B.SPEC_OK
    assert lib.spec_tree_attention_shared(ctypes.byref(s), None, 0, None) == B.SPEC_OK


def test_workspaces_are_checked(lib):
    p = _fill(B.SpecBeamReorderParams(), **REORDER)
    size = lib.spec_beam_reorder_workspace_size(ctypes.byref(p))
    assert size > 0 and size % 256 == 0
    for ws, n in ((None, size), (FAKE, size - 1), (FAKE + 16, size)):
        assert lib.spec_beam_reorder(ctypes.byref(p), ws, n, None) == INV


def test_binding_refuses_cpu_tensors():
    z, f, i = torch.zeros(2, 2, 16, 128), torch.zeros(2, 3), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        B.attention_window_params(z, z, z, i, i, i, i, 1, 4, 0, z, None, i)
    with pytest.raises(ValueError, match="CUDA"):
        B.attention_shared_params(z, z, z, i, i, i, i, 1, i, i, z, None, i)
    with pytest.raises(ValueError, match="CUDA"):
        B.beam_select_params(f, 3, 1.0, f, i, i, 0, 0.0, i, i, f, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        B.beam_reorder_params(z, z, i, i, i, i)
