"""Limits of windowed and shared-prefix attention that are checked before any CUDA call."""
import ctypes

import pytest

from speculative_decoding_draft_tree_gb300 import binding as B
from speculative_decoding_draft_tree_gb300 import build
from test_span_beam_library import ATTN, FAKE, UNS, _fill


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return B.load_library()


@pytest.mark.parametrize("T_max,H_q,code", [(256, 8192, UNS), (256, 8191, 0), (1, 65535 * 32 + 1, UNS), (1, 65535 * 32, 0)])
def test_query_rows_beyond_the_merges_grid_are_refused(lib, T_max, H_q, code):
    """A request's rows under a KV head, 32 a CTA.  What is allowed has a workspace; nothing is launched."""
    w, s = B.SpecAttnWindowParams(), B.SpecAttnSharedParams()
    for p in (w, s):
        _fill(p.attn, **{**ATTN, **dict(T_max=T_max, H_q=H_q, H_kv=1)})
    w.window, s.num_groups, s.group_offset, s.shared_len = 1, 2, FAKE, FAKE
    sizes = (lib.spec_attention_window_workspace_size(ctypes.byref(w)), lib.spec_attention_shared_workspace_size(ctypes.byref(s)))
    if code:
        assert sizes == (0, 0)
        assert lib.spec_tree_attention_window(ctypes.byref(w), FAKE, 1 << 60, None) == code
        assert lib.spec_tree_attention_shared(ctypes.byref(s), FAKE, 1 << 60, None) == code
    else:
        assert min(sizes) > 0
