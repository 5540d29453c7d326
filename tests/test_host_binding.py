"""Which tensors csrc/binding.cpp takes: ordinary ones.  A tensor that torch's
function transforms make has a shape and a device but no memory of its own, and
asking for its address raises."""

import pytest
import torch

from exact_io_aware_order_gb300 import _lib, build


@pytest.fixture(scope="module")
def takes():
    build.build()
    return _lib.binding().takes


def seen_inside(transform):
    """The tensor that a transformed function is handed."""
    got = []

    def f(x):
        assert type(x) is torch.Tensor
        got.append(x)
        return x.sum()

    transform(f)(torch.zeros(4, 2, 3))
    return got[0]


def test_takes_ordinary_tensors(takes):
    x = torch.zeros(4, 2, 3)
    assert takes(x) and takes(x[1:]) and takes(x.transpose(0, 1)) and takes(torch.empty(0))
    assert takes(x.requires_grad_())


@pytest.mark.parametrize("transform", [torch.vmap, torch.func.grad])
def test_leaves_tensors_without_memory(takes, transform):
    assert not takes(seen_inside(transform))


def test_leaves_subclasses_and_other_objects(takes):
    class Sub(torch.Tensor):
        pass

    for x in (torch.zeros(2).as_subclass(Sub), None, 3, [torch.zeros(2)]):
        assert not takes(x)
