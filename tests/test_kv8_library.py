"""Host side of the 8-bit cache's entry points: struct layouts and refusals, before any CUDA call."""
import ctypes
import subprocess

import pytest
import torch

from speculative_decoding_draft_tree_gb300 import binding as B
from speculative_decoding_draft_tree_gb300 import build

FAKE = 0x100000   # 16-byte aligned, never dereferenced: validation fails first
INV, UNS = B.SPEC_ERR_INVALID_ARG, B.SPEC_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return B.load_library()


def test_struct_layouts_match_header(tmp_path):
    structs = {"spec_kv8_append_params": B.SpecKv8AppendParams, "spec_attn_kv8_params": B.SpecAttnKv8Params,
               "spec_kv8_compact_params": B.SpecKv8CompactParams, "spec_fork_params": B.SpecForkParams}
    lines, want = ["#include <stdio.h>", "#include <stddef.h>", '#include "spec_verify.h"', "int main(void) {"], []
    for cname, py in structs.items():
        lines.append(f'  printf("%zu\\n", sizeof({cname}));')
        want.append(ctypes.sizeof(py))
        for f, _ in py._fields_:
            lines.append(f'  printf("%zu\\n", offsetof({cname}, {f}));')
            want.append(getattr(py, f).offset)
    lines += ['  printf("%d\\n", (int)SPEC_E4M3);', "  return 0;", "}"]
    want.append(B.SPEC_E4M3)
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


CACHE = dict(B=2, H_kv=2, head_dim=128, block_size=16, num_blocks=8, max_blocks_per_req=4)
BAD_CACHE = [(dict(B=0), INV), (dict(H_kv=0), INV), (dict(head_dim=0), INV), (dict(block_size=0), INV), (dict(num_blocks=0), INV),
             (dict(max_blocks_per_req=0), INV), (dict(k_cache=None), INV), (dict(v_cache=FAKE + 8), INV), (dict(k_scale=None), INV),
             (dict(v_scale=None), INV), (dict(block_table=None), INV), (dict(req_status=None), INV), (dict(head_dim=120), UNS),
             (dict(head_dim=272), UNS), (dict(block_size=1025), UNS), (dict(num_blocks=1 << 30), UNS),
             (dict(max_blocks_per_req=1 << 30), UNS)]


@pytest.mark.parametrize("change,code", BAD_CACHE + [
    (dict(dtype=2), INV), (dict(dtype=-1), INV), (dict(N=-1), INV), (dict(k_new=None), INV), (dict(v_new=FAKE + 2), INV),
    (dict(k_ld=255), INV), (dict(v_ld=260), INV), (dict(start=None), INV), (dict(row_offset=None), INV)])
def test_append_refusals(lib, change, code):
    p = _fill(B.SpecKv8AppendParams(), **{**CACHE, **dict(dtype=1, N=4, k_ld=256, v_ld=256), **change})
    assert lib.spec_kv8_append(ctypes.byref(p), None) == code


@pytest.mark.parametrize("change,code", BAD_CACHE + [
    (dict(dtype=2), INV), (dict(N=-1), INV), (dict(T_max=0), INV), (dict(T_max=257), INV), (dict(H_q=3), INV), (dict(H_q=0), INV),
    (dict(q=None), INV), (dict(o=FAKE + 4), INV), (dict(anc_mask=None), INV), (dict(prefix_len=None), INV),
    (dict(node_offset=None), INV)])
def test_attention_refusals(lib, change, code):
    p = _fill(B.SpecAttnKv8Params(), **{**CACHE, **dict(dtype=1, N=4, T_max=2, H_q=4), **change})
    assert lib.spec_tree_attention_kv8(ctypes.byref(p), FAKE, 1 << 40, None) == code
    assert lib.spec_attention_kv8_workspace_size(ctypes.byref(p)) == 0


@pytest.mark.parametrize("change,code", BAD_CACHE + [
    (dict(num_layers=0), INV), (dict(num_layers=65536), UNS), (dict(max_path=0), INV), (dict(layer_stride=-16), INV),
    (dict(layer_stride=24), INV), (dict(scale_layer_stride=-1), INV), (dict(path=None), INV), (dict(n_acc=None), INV),
    (dict(slot_map=None), INV), (dict(new_kv_len=None), INV), (dict(blocks_in_use=None), INV), (dict(prefix_len=None), INV)])
def test_compact_refusals(lib, change, code):
    p = _fill(B.SpecKv8CompactParams(), **{**CACHE, **dict(num_layers=1, max_path=4, layer_stride=0, scale_layer_stride=0), **change})
    assert lib.spec_kv8_compact(ctypes.byref(p), None) == code


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), INV), (dict(B=0), INV), (dict(F=-1), INV), (dict(num_layers=0), INV), (dict(num_layers=65536), UNS),
    (dict(head_dim=8), INV), (dict(layer_stride=8), INV), (dict(k_cache=None), INV), (dict(v_cache=FAKE + 4), INV),
    (dict(k_scale=None), INV), (dict(block_table=None), INV), (dict(kv_len=None), INV), (dict(src=None), INV), (dict(dst=None), INV),
    (dict(new_block=None), INV), (dict(fork_status=None), INV), (dict(block_size=1 << 30), UNS)])
def test_fork_refusals(lib, change, code):
    p = _fill(B.SpecForkParams(), **{**CACHE, **dict(dtype=2, F=1, num_layers=1, layer_stride=0, scale_layer_stride=0), **change})
    assert lib.spec_kv_fork(ctypes.byref(p), None) == code


def test_null_and_empty_calls(lib):
    for f in (lib.spec_kv8_append, lib.spec_kv8_compact, lib.spec_kv_fork):
        assert f(None, None) == INV
    assert lib.spec_tree_attention_kv8(None, None, 0, None) == INV
    p = _fill(B.SpecKv8AppendParams(), **{**CACHE, **dict(dtype=1, N=0, k_ld=256, v_ld=256, k_new=None, v_new=None)})
    assert lib.spec_kv8_append(ctypes.byref(p), None) == B.SPEC_OK
    p = _fill(B.SpecAttnKv8Params(), **{**CACHE, **dict(dtype=1, N=0, T_max=2, H_q=4, q=None, o=None, anc_mask=None)})
    assert lib.spec_tree_attention_kv8(ctypes.byref(p), None, 0, None) == B.SPEC_OK
    p = _fill(B.SpecForkParams(), **{**CACHE, **dict(dtype=1, F=0, num_layers=1, layer_stride=0, src=None, dst=None,
                                                    new_block=None, fork_status=None, k_scale=None)})
    assert lib.spec_kv_fork(ctypes.byref(p), None) == B.SPEC_OK


def test_binding_refuses_cpu_tensors_and_wrong_types():
    z = torch.zeros(2, 2, 16, 128, dtype=torch.uint8)
    s = torch.zeros(2, 2)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        B.kv8_append_params(s, s, z, z, s, s, i, i, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_fork_params(z, z, i, i, i, i, i, i, s, s)
