"""The AdamW optimizer as an object: its options, copies of it, what it refuses.  CPU only."""
import copy
import io
import pickle

import pytest
import torch

from aware_conv_amd import AdamW

OPTIONS = {"bits": 8, "master": False, "max_norm": 0.5, "skip_nonfinite": True, "grad_scale": 0.25}


def saved_and_loaded(opt):
    f = io.BytesIO()
    torch.save(opt, f)
    f.seek(0)
    return torch.load(f, weights_only=False)  # what this test has just written


@pytest.mark.parametrize("copied", [copy.deepcopy, lambda o: pickle.loads(pickle.dumps(o)), saved_and_loaded])
def test_copies_have_the_options(copied):
    opt = AdamW([torch.nn.Parameter(torch.ones(3))], lr=0.1, **OPTIONS)
    opt.grad_scale = 0.125  # an attribute that a training loop sets
    other = copied(opt)
    for n, v in dict(OPTIONS, grad_scale=0.125).items():
        assert getattr(other, n) == v, n
    assert other.param_groups[0]["lr"] == 0.1
    assert other.step() is None  # nothing has a gradient
