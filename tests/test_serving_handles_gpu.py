"""The cache's handle: copies of it, and tensors put in place of its own."""
import copy
import io

import pytest
import torch

import exact_io_aware_52_b200 as fa
from tests import serving_ref as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def dev():
    return torch.device("cuda:0")


def a_cache():
    return fa.PagedCache(*(t.to(dev()) for t in ref.pool(60, [20, 33], 2, 16, 64)))


def through_a_file(x):
    f = io.BytesIO()
    torch.save(x, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


@pytest.mark.parametrize("how", [copy.deepcopy, through_a_file])
def test_copies_of_a_cache_are_apart(how):
    """A copy's calls read and write the copy's tensors, and leave those it was made from."""
    c = a_cache()
    mine = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale, c.table)]
    other = how(c)
    x = torch.randn(2, 2, 3, 64, generator=torch.Generator().manual_seed(61)).to(BF16).to(dev())
    start = torch.tensor([17, 30], dtype=torch.int32, device=dev())
    fa.cache_append(other, x, x, start)
    for t, want in zip((c.k, c.v, c.k_scale, c.v_scale, c.table), mine):
        assert torch.equal(t.view(torch.uint8), want.view(torch.uint8))
    fa.cache_append(c, x, x, start)
    for a, b in zip((c.k, c.v, c.k_scale, c.v_scale), (other.k, other.v, other.k_scale, other.v_scale)):
        assert a.data_ptr() != b.data_ptr() and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_a_shallow_copy_shares_the_tensors():
    c = a_cache()
    other = copy.copy(c)
    n = torch.tensor([20, 33], dtype=torch.int32, device=dev())
    assert other.k is c.k
    assert all(torch.equal(a, b) for a, b in zip(fa.cache_gather(c, n, 33), fa.cache_gather(other, n, 33)))


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "table", "page", "n_pages"])
def test_a_cache_refuses_other_tensors(name):
    """Calls use the places that were checked when the cache was made."""
    c = a_cache()
    value = getattr(c, name)
    with pytest.raises(AttributeError):
        setattr(c, name, value.clone() if torch.is_tensor(value) else value)


class Layer(fa.PagedCache):
    """A program's own cache, with more than the package's."""

    def __init__(self, index):
        super().__init__(*(t.to(dev()) for t in ref.pool(62, [20], 1, 16, 64)))
        self.index = index


def test_a_cache_can_have_more():
    c = Layer(7)
    c.note = [1, 2]
    for other in (copy.copy(c), copy.deepcopy(c)):
        assert type(other) is Layer and other.index == 7 and other.note == [1, 2]
        n = torch.tensor([20], dtype=torch.int32, device=dev())
        assert all(torch.equal(a, b) for a, b in zip(fa.cache_gather(c, n, 20), fa.cache_gather(other, n, 20)))
    c.index = 8
