"""A group's handle belongs to one object, which frees it: copies are refused (no GPU)."""

import copy
import pickle

import pytest

import matrix_optimizer_step_02_amd as mo


@pytest.mark.parametrize("kind", ["RotatedAdamGroup", "AdamWGroup"])
@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, pickle.dumps])
def test_groups_are_not_copied(kind, how):
    cls = getattr(mo, kind)
    group = cls.__new__(cls)
    group.params = []
    with pytest.raises(TypeError, match="another group"):
        how(group)
