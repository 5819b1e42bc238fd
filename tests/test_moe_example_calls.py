"""The decoding step of examples/moe_layer.py is four calls of the library and nothing else on the
GPU, given the slots' numbers.  No GPU needed: the calls are replaced by ones that record themselves."""
import importlib.util
import os
import types

import torch

from tests.test_abi_moe_layer import ROOT, lib  # noqa: F401  (lib is the fixture)


def test_decode_is_four_calls(lib, monkeypatch):  # noqa: F811
    spec = importlib.util.spec_from_file_location(
        "moe_layer_example_calls", os.path.join(ROOT, "examples", "moe_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    calls = []

    def record(name, result):
        def call(*args):
            calls.append((name, args))
            return result
        return call

    monkeypatch.setattr(example, "hg", types.SimpleNamespace(
        hg_router_topk=record("router", ("ids", "weights")),
        hg_expert_matvec_swiglu=record("gate_up", "h"), hg_expert_matvec=record("down", "y"),
        hg_combine_topk=record("combine", "out")))
    experts = types.SimpleNamespace(gate_up=("gu", "gus"), down=("dn", "dns"))
    slots = example.slot_numbers(3, 2, "cpu")
    assert slots.tolist() == list(range(6)) and slots.dtype == torch.int32
    x = types.SimpleNamespace()                             # nothing but the calls may touch it
    assert example.decode(x, "logits", 2, experts, slots) == "out"
    assert [name for name, _ in calls] == ["router", "gate_up", "down", "combine"]
    assert calls[3][1] == ("y", slots, "weights")
