"""The layers' plain projections on the CPU: whatever view they are given, one
matrix product.  torch takes a product of a three-dimensional view whose rows
do not follow each other (a window behind its persistent rows, the second
half of an output) as a batched one with the weight as a transposed operand
of batch distance 0, which in bf16 has read out of bounds on a GPU."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from test_trained_neural_amd.attention import _product


class Products(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.seen = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if "mm" in str(func):
            self.seen.append(str(func))
        return func(*args, **(kwargs or {}))


VIEWS = {"whole": lambda t: t, "behind the first rows": lambda t: t[:, 4:], "one entry": lambda t: t[1:2, 4:],
         "one token": lambda t: t[:, 5:6], "shared": lambda t: t[:1].expand(3, -1, -1),
         "half of an output": lambda t: t.unflatten(2, (4, 16))[:, 10:].flatten(2),
         "tokens first": lambda t: t.transpose(0, 1), "no tokens": lambda t: t[:, :0], "rows": lambda t: t[0]}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("view", list(VIEWS))
def test_projections_are_single_products(view, dtype):
    rand = lambda seed, *n: torch.randn(*n, generator=torch.Generator().manual_seed(seed)).to(dtype)  # noqa: E731
    x, w = VIEWS[view](rand(1, 3, 20, 64)), rand(2, 48, 64)
    with Products() as seen:
        y = _product(x, w)
    assert not any("bmm" in s for s in seen.seen), seen.seen
    assert y.shape == x.shape[:-1] + (48,) and y.is_contiguous() and y.dtype == dtype
    # sums of 64 products in fp32 and one rounding
    want = x.double() @ w.double().t()
    size = x.double().abs() @ w.double().abs().t()
    assert bool(((y.double() - want).abs() <= size * 64 * 2.0 ** -24 + want.abs() * torch.finfo(dtype).eps / 2).all())
