"""Copies of a Rotary: of the object, of a model that holds it, and through a file (no GPU)."""

import copy
import io
import pickle

import pytest
import torch

from matrix_optimizer_step_02_amd import train


def through_a_file(rope):
    f = io.BytesIO()
    torch.save(rope, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


class Layer(torch.nn.Module):
    def __init__(self, rope):
        super().__init__()
        self.rope = rope


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r)), through_a_file,
                                 lambda r: copy.deepcopy(Layer(r)).rope])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_a_copy_turns_as_the_original(how, layout):
    rope = train.Rotary([1.0, 0.5, 0.1], layout=layout, scale=1.25, device="cpu")
    got = how(rope)
    assert type(got) is train.Rotary
    assert torch.equal(got.turns, rope.turns) and got[1:5] == rope[1:5]
    assert got.ptr == got.turns.data_ptr()
    assert got.c(None, 3, (1, 2, 2, 8), torch.device("cpu")).turns == got.ptr
