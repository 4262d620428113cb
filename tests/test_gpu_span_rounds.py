"""Groups of requests as inputs of a round: twins and pipelines of a VerifyStep under shared prefixes."""
import pytest
import torch

import kv8_util as U
from speculative_decoding_draft_tree_gb300 import workloads as W
from speculative_decoding_draft_tree_gb300.api import RoundPipeline, VerifyStep

pytestmark = pytest.mark.gpu


def _workload():
    """Requests whose first pages are the same, the caches' restoring, and the plain round's tokens."""
    w = W.make_config(4, scale="small", device="cuda")
    bs = w.k_cache.shape[3]
    P = int(w.prefix_len.min()) // bs * bs
    w.block_table[:, :P // bs] = w.block_table[0, :P // bs].clone()
    caches = (w.k_cache.clone(), w.v_cache.clone())

    def again():
        w.k_cache.copy_(caches[0])
        w.v_cache.copy_(caches[1])

    plain = VerifyStep(w)
    plain.run()
    torch.cuda.synchronize()
    return w, P, again, (plain.out_tokens.clone(), plain.out_len.clone())


def test_a_twin_has_groups_of_its_own():
    w, P, again, want = _workload()
    step = VerifyStep(w)
    step.enable_shared(U.ints([0, w.B]), U.ints([P]))
    a, b = step.twin(), step.twin()
    b.step_input_tensors()["shared_len"].fill_(1 << 20)          # beyond every prefix
    for s, status in ((b, 2), (a, 0), (step, 0)):
        again()
        s.run()
        torch.cuda.synchronize()
        assert s.req_status.tolist() == [status] * w.B
        if status == 0:
            assert torch.equal(s.out_tokens, want[0]) and torch.equal(s.out_len, want[1])


def test_a_pipelines_rounds_bring_their_groups():
    w, P, again, want = _workload()
    step = VerifyStep(w)
    step.enable_shared(U.ints([0, w.B, w.B]), U.ints([P, 0]))
    pipe = RoundPipeline(step)
    mine = pipe.steps[0].step_input_tensors()
    packs = {"one": pipe.pinned_host_inputs()}
    mine["group_offset"].copy_(U.ints([0, 1, w.B]))
    mine["shared_len"].copy_(U.ints([0, P]))
    packs["two"] = pipe.pinned_host_inputs()
    mine["shared_len"].fill_(1 << 20)
    packs["bad"] = pipe.pinned_host_inputs()
    torch.cuda.synchronize()
    for name in ("one", "two", "bad", "two", "one", "bad", "one"):
        again()
        i = pipe.submit(packs[name])
        pipe.finish()
        torch.cuda.synchronize()
        assert pipe.steps[i % 2].req_status.tolist() == [2 if name == "bad" else 0] * w.B
        if name != "bad":
            out = pipe.host_outputs(i)
            assert torch.equal(out["out_tokens"], want[0].cpu()) and torch.equal(out["out_len"], want[1].cpu())


def test_a_step_takes_one_form_once():
    w, P, _, _ = _workload()
    for first in ("window", "shared"):
        step = VerifyStep(w)
        if first == "window":
            step.enable_window(100, 2)
        else:
            step.enable_shared(U.ints([0, w.B]), U.ints([P]))
        for call in (lambda: step.enable_window(100, 2), lambda: step.enable_shared(U.ints([0, w.B]), U.ints([P]))):
            with pytest.raises(ValueError, match="once"):
                call()
