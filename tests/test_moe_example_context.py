"""What the forward pass of examples/moe_layer.py keeps for the backward: the experts' FP8 inputs
only where the experts learn.  No GPU needed: the library's calls are replaced."""
import importlib.util
import os
import types

import pytest
import torch

from tests.test_abi_moe_layer import ROOT, lib  # noqa: F401  (the fixture)


@pytest.fixture
def example(lib, monkeypatch):  # noqa: F811
    spec = importlib.util.spec_from_file_location(
        "moe_layer_example_context", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.wgrads = []

    def gives(*names):
        return lambda *a, **kw: names if len(names) > 1 else names[0]

    t = torch.zeros(6, 4, dtype=torch.bfloat16)
    monkeypatch.setattr(m, "hg", types.SimpleNamespace(
        hg_router_topk=gives("ids", "weights"), hg_plan_expert_offsets=gives("off", "src", "place"),
        hg_quantize_scatter_acts=gives("a", "a_scale"), hg_dispatch_acts=gives("a", "a_scale"),
        hg_grouped_w4a8_gemm=lambda *a: t, hg_swiglu_quantize=gives("h", "h_scale", "z8", "z8_scale"),
        hg_combine_topk=gives(torch.zeros(3, 4)), hg_combine_topk_bwd=gives("dy", "dw"),
        hg_swiglu_bwd=gives("dz"), hg_dispatch_tokens_bwd=gives("dx", None),
        hg_router_topk_bwd=lambda *a: torch.zeros(3, 2),
        hg_rmsnorm_quantize=gives(torch.zeros(3, 4), "n8", "n8_scale", torch.zeros(3, 4), "rstd"),
        hg_rmsnorm_bwd=gives("dx", "dgain"),
        hg_grouped_wgrad_fp8=lambda *a: m.wgrads.append(a) or f"grad {len(m.wgrads)}"))
    return m


EXPERTS = types.SimpleNamespace(gate_up=(1, 1), down=(2, 2), gate_up_t=(3, 3), down_t=(4, 4))
KEPT = {"a", "a_scale", "h", "h_scale"}


def _held(ctx):
    held = set()
    for c in ctx:
        held |= _held(c) if isinstance(c, tuple) else {c} if isinstance(c, str) else set()
    return held


def test_frozen_experts_inputs_are_not_kept(example, monkeypatch):
    logits = torch.zeros(3, 2)
    contexts = []
    forward = example.forward
    monkeypatch.setattr(example, "forward", lambda *a, **kw: contexts.append(forward(*a, **kw)) or
                        contexts[-1])
    example.train_step("x", logits, "dout", 2, EXPERTS)
    assert not _held(contexts[0][1]) & KEPT and {"z8", "z8_scale"} <= _held(contexts[0][1])
    assert forward("x", logits, 2, EXPERTS, keep=False)[1] is None
    assert not example.wgrads


def test_learning_experts_inputs_are_kept(example):
    dout = torch.zeros(3, 4)
    example.hg.hg_dispatch_tokens_bwd = lambda *a: (torch.zeros(3, 4), None)
    out = example.train_block(torch.zeros(3, 4), None, None, torch.zeros(4, 2), dout, 2, EXPERTS)
    assert out[-1] == ("grad 1", "grad 2")
    assert example.wgrads == [("dz", "a", "a_scale", "off"), ("dy", "h", "h_scale", "off")]


def test_weight_gradients_want_what_they_need(example):
    _, ctx = example.forward("x", torch.zeros(3, 2), 2, EXPERTS)
    with pytest.raises(AssertionError):
        example.backward("dout", ctx, 2, EXPERTS, weight_grads=True)
