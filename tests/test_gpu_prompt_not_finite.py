"""Prompt attention over values of which many are not finite, where the rows of a tile see different numbers of them."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_gpu_prompt import check, dev, randn, starts_of, zg  # noqa: E402, F401 (zg and dev are fixtures)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim, Hq, Hk", [(32, 2, 2), (64, 3, 1), (96, 6, 2), (128, 2, 1), (128, 5, 1)])
def test_many_values_that_are_not_finite(zg, dev, dtype, dim, Hq, Hk):  # noqa: F811
    """A third of the rows of values hold a NaN or an infinity in one of three dims; the others of the dims are as if
    there were none."""
    lengths = [300, 1, 0, 129, 517]
    T = sum(lengths)
    q, k, v = (randn((T, h, dim), dtype, 3 + h + dim) for h in (Hq, Hk, Hk))
    g = torch.Generator(device="cuda").manual_seed(dim)
    pick = torch.randint(0, 9, (T, Hk), generator=g, device="cuda")
    for i, (d, x) in enumerate(((3, math.nan), (dim // 2 + 1, math.inf), (dim - 1, -math.inf))):
        v[:, :, d] = torch.where(pick == i, torch.full_like(v[:, :, d], x), v[:, :, d])
    for causal in (True, False):
        check(zg, dev, q, k, v, starts_of(lengths), causal)
