"""GPU tests of several verification rounds over the 8-bit cache, one after the other."""
import dataclasses

import pytest
import torch

from speculative_decoding_draft_tree_gb300.api import RoundPipeline, VerifyStep, _packed
from test_gpu_kv8 import _round_case

pytestmark = pytest.mark.gpu


def _bytes(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("cid", [2, 4])
def test_pipelined_rounds_append_the_rows_of_their_own_round(cid):
    """Five rounds submitted without a wait in between, each with new K/V rows and a new q, against run()
    round by round: the results and the cache's bits."""
    w, step, (k, v, ks, vs, k_new, v_new) = _round_case(cid, 2)
    cache, before = (k, v, ks, vs), [t.clone() for t in (k, v, ks, vs)]
    g = torch.Generator(device="cuda").manual_seed(5)
    rounds = [{n: torch.randn(t.shape, generator=g, device="cuda").to(t.dtype) * (i + 1)
               for n, t in (("k_new", k_new), ("v_new", v_new), ("q", w.q))} for i in range(5)]
    want, caches = [], []
    for x in rounds:
        for n, t in (("k_new", k_new), ("v_new", v_new), ("q", w.q)):
            t.copy_(x[n])
        step.run()
        torch.cuda.synchronize()
        want.append([t.cpu().clone() for t in (step.o, step.out_tokens, step.new_kv_len)])
        caches.append([t.clone() for t in cache])
    for t, b in zip(cache, before):
        t.copy_(b)
    assert not any(torch.equal(_bytes(a[0]), _bytes(b[0])) for a, b in zip(caches, caches[1:]))
    pipe = RoundPipeline(step)
    hosts = []
    for x in rounds:
        buf, views = _packed(step.step_input_tensors(), "cpu", pin=True)
        buf.copy_(pipe.pinned_host_inputs()["_pack"])
        for n, t in x.items():
            views[n].copy_(t)
        hosts.append({"_pack": buf})
    k_new.fill_(float("nan"))                   # the pipeline's steps have rows of their own
    v_new.fill_(float("nan"))
    torch.cuda.synchronize()
    for i, h in enumerate(hosts):
        pipe.submit(h)
    pipe.finish()
    torch.cuda.synchronize()
    for i in (3, 4):
        out = pipe.host_outputs(i)
        assert torch.equal(out["out_tokens"], want[i][1]) and torch.equal(out["new_kv_len"], want[i][2])
        assert torch.equal(_bytes(pipe.steps[i % 2].o.cpu()), _bytes(want[i][0]))
    for t, c in zip(cache, caches[-1]):
        assert torch.equal(_bytes(t), _bytes(c))


def test_run_from_host_brings_the_new_rows():
    w, step, (k, v, ks, vs, k_new, v_new) = _round_case(2, 1)
    before = [t.clone() for t in (k, v, ks, vs)]
    step.run()
    torch.cuda.synchronize()
    want = [t.clone() for t in (k, v, ks, vs)] + [step.o.clone()]
    host = step.pinned_host_inputs()
    assert {"k_new", "v_new"} <= set(host)
    for t, b in zip((k, v, ks, vs), before):
        t.copy_(b)
    k_new.zero_()
    v_new.zero_()
    step.run_from_host(host, step.host_output_buffers())
    torch.cuda.synchronize()
    for t, x in zip((k, v, ks, vs, step.o), want):
        assert torch.equal(_bytes(t), _bytes(x))


def test_a_round_over_the_8_bit_cache_needs_no_16_bit_one():
    """The workload's own cache may be a page of its shape: with enable_kv8 nothing reads it."""
    w, step, (k, v, ks, vs, k_new, v_new) = _round_case(4, 2)
    before = [t.clone() for t in (k, v, ks, vs)]
    step.run()
    torch.cuda.synchronize()
    names = ("o", "lse", "out_tokens", "out_len", "path", "n_acc", "new_kv_len", "slot_map", "req_status")
    want = [getattr(step, n).clone() for n in names] + [t.clone() for t in (k, v, ks, vs)]
    for t, b in zip((k, v, ks, vs), before):
        t.copy_(b)
    page = torch.full_like(w.k_cache[:1, :1], float("nan"))
    small = VerifyStep(dataclasses.replace(w, k_cache=page, v_cache=page.clone()))
    small.enable_kv8(k, v, ks, vs, k_new, v_new)
    for s in (small, small.twin()):
        for t, b in zip((k, v, ks, vs), before):
            t.copy_(b)
        s.run()
        torch.cuda.synchronize()
        for t, x in zip([getattr(s, n) for n in names] + [k, v, ks, vs], want):
            assert torch.equal(_bytes(t), _bytes(x))
