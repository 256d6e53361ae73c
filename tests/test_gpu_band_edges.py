"""The band attention and the query/key norm where they can go wrong beyond the sizes of
tests/test_gpu_band.py: scores far from zero, non-finite inputs, large head groups, units of
several tokens, gradients that are not wanted.  References are plain 64-bit forms; each bound is
derived where it is used."""
import pytest
import torch

from test_gpu_band import DTYPES, case, compare, dcn, make, run  # noqa: F401  (dcn is a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


# One active key tile a half in grad_q's second pass over the keys: nothing but the kernel's own barriers
# orders the exchange of a row's sum before it and the one behind it.
ONE_TILE = [
    case("f16", 2, 200, 60, 4, 4, 64),                       # 60 keys
    case("bf16", 1, 512, 512, 8, 2, 128, right=0),           # the first CTAs of a causal band with shared heads
    case("f16", 1, 300, 300, 4, 1, 32, right=0, nb=8, M=16),
]


# Rings of two and three slots with many tiles behind them: grad_q's halves may be as far apart as the ring.
RINGS = [
    case("bf16", 1, 700, 700, 4, 2, 128, nb=8, M=16),
    case("f16", 2, 300, 900, 4, 4, 72, left=500, right=0),
]


@pytest.mark.parametrize("c", ONE_TILE + RINGS, ids=str)
def test_order_within_grad_q(dcn, c):  # noqa: F811
    """Equal to the definition and the same from call to call."""
    t = make(c, 3)
    first = compare(dcn, c, t)
    for _ in range(20):
        for x, y in zip(first, run(dcn, c, t)):
            assert x is y is None or torch.equal(x, y)
