"""The training products' binding refuses an input that is missing, rather than
taking a fresh buffer for it (on the CPU: the library's entry points and the
device are stood in for)."""
import types
import unittest.mock as mock

import pytest
import torch

import mixture_experts_layer_61_b200 as moe

T, H, E, K, I = 32, 64, 4, 2, 128


@pytest.fixture
def calls(monkeypatch):
    """Tensors on the CPU pass as the current device's; the library's calls are counted, not made."""
    made = mock.Mock(return_value=0)
    names = ("moe_grouped_gate_up_train", "moe_grouped_down_grad", "moe_grouped_gate_up_grad",
             "moe_grouped_down_wgrad", "moe_grouped_gate_up_wgrad")
    fake = types.SimpleNamespace(**{n: made for n in names},
                                 moe_padded_rows_max=moe.lib().moe_padded_rows_max)
    monkeypatch.setattr(moe, "lib", lambda: fake)
    monkeypatch.setattr(moe, "_dev", lambda: torch.device("cpu"))
    monkeypatch.setattr(moe, "_raw_stream", lambda dev: 0)
    return made


def arguments(name):
    """(the call's tensors by place, the places of its row inputs)"""
    c = moe.config(T, H, E, K, I)
    bf = torch.bfloat16
    R = moe.padded_rows_max(c)
    row = lambda n: torch.zeros((R, n), dtype=bf)
    off, ws = torch.zeros(E + 1, dtype=torch.int32), torch.zeros(1024, dtype=torch.uint8)
    w13, w2 = torch.zeros((E, 2 * I, H), dtype=bf), torch.zeros((E, H, I), dtype=bf)
    return {
        "grouped_gate_up_train": ([c, row(H), w13, off, ws], (1,)),
        "grouped_down_grad": ([c, row(H), w2, row(2 * I), off, ws], (1, 3)),
        "grouped_gate_up_grad": ([c, row(2 * I), w13, off, ws], (1,)),
        "grouped_down_wgrad": ([c, row(H), row(I), off, ws], (1, 2)),
        "grouped_gate_up_wgrad": ([c, row(2 * I), row(H), off, ws], (1, 2)),
    }[name]


@pytest.mark.parametrize("name", ["grouped_gate_up_train", "grouped_down_grad", "grouped_gate_up_grad",
                                  "grouped_down_wgrad", "grouped_gate_up_wgrad"])
def test_a_missing_input_is_refused(calls, name):
    args, inputs = arguments(name)
    getattr(moe, name)(*args)  # complete: made once
    assert calls.call_count == 1
    for i in inputs:
        with pytest.raises(ValueError, match="must be given"):
            getattr(moe, name)(*[None if j == i else a for j, a in enumerate(args)])
    assert calls.call_count == 1
