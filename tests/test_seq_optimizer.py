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


@pytest.mark.parametrize("kw", [{"lr": -1e-3}, {"eps": -1e-8}, {"weight_decay": -0.1}, {"lr": float("nan")},
                                {"eps": float("nan")}, {"weight_decay": float("inf")}, {"lr": float("inf")}])
def test_values_that_mean_nothing(kw):
    w = torch.nn.Parameter(torch.zeros(3))
    with pytest.raises(ValueError, match=list(kw)[0]):
        AdamW([w], **kw)
    with pytest.raises(ValueError, match=list(kw)[0]):
        AdamW([dict(params=[w], **kw)])
    opt = AdamW([torch.nn.Parameter(torch.zeros(2))])
    with pytest.raises(ValueError, match=list(kw)[0]):
        opt.add_param_group(dict(params=[w], **kw))
    assert len(opt.param_groups) == 1
    AdamW([w], lr=torch.tensor(-1.0))  # a device value is not looked at


def test_strided_parameters_are_refused_when_they_are_given():
    w = torch.nn.Parameter(torch.zeros(2, 3, 4, 4).to(memory_format=torch.channels_last))
    with pytest.raises(ValueError, match="contiguous"):
        AdamW([w])


def test_other_mistakes_are_told_as_by_the_base_class():
    opt = AdamW([torch.nn.Parameter(torch.zeros(2))])
    with pytest.raises(TypeError, match="must be a dict"):
        opt.add_param_group([torch.nn.Parameter(torch.zeros(2))])
    with pytest.raises(ValueError, match="more than one parameter group"):
        opt.add_param_group({"params": opt.param_groups[0]["params"]})
