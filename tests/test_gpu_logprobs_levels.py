"""k3moe_logprobs on logits away from 0: the results of a row do not depend on
where it stands."""
import numpy as np
import pytest
import torch

from test_gpu_logprobs import DEV, _check, _ids, _run, _x

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]


@pytest.mark.parametrize("offset", [-30000.0, -3000.0, -100.0, 100.0, 3000.0, 30000.0])
@pytest.mark.parametrize("T,V", [(3, 20000), (600, 9000)])
def test_entropy_away_from_zero(T, V, offset):
    _check(_x(T, V, seed=3) + offset, _ids(T, V, 2), 4)


@pytest.mark.parametrize("offset", [-65536.0, -1024.0, 1.0, 100.0, 30000.0, 65536.0])
@pytest.mark.parametrize("T,V", [(3, 20000), (600, 9000)])
def test_a_shifted_row_has_the_same_bits(T, V, offset):
    """Multiples of 2^-6 below 2^17 are fp32 numbers, so the shift and every x - max are exact."""
    x = (_x(T, V, seed=5) * 64).round() / 64
    ids = _ids(T, V, 2)
    moved = x + offset
    assert torch.equal(moved - offset, x)
    for a, b in zip(_run(x, ids, 7), _run(moved, ids, 7)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("level", [1e5, 1e6, 1e7, 1e8, 1e15, 1e30, 2.5e38])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("T", [2, 600])
def test_neighbouring_numbers_at_any_level(T, sign, level):
    """Rows whose logits are a few steps of fp32 apart."""
    V = 9000
    step = float(np.spacing(np.float32(level)))
    at = torch.randint(-3, 4, (T, V), generator=torch.Generator().manual_seed(7)).to(DEV)
    x = (sign * level + step * at.double()).float()
    _check(x, _ids(T, V, 2), 5)


LOWEST = [float(np.finfo(np.float32).min), float(torch.finfo(torch.bfloat16).min), -1e30, -1e20, -1e10, -65504.0]


@pytest.mark.parametrize("fill", LOWEST)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [6, 600])
def test_tokens_banned_by_the_lowest_numbers(T, dtype, fill):
    """Whole chunks of 4096 and 8192 of them, the first, the last, all but one, all: as valid as any other row."""
    if dtype == torch.bfloat16 and fill < torch.finfo(dtype).min:
        pytest.skip("not a number of this type")
    V = 20000
    x = _x(T, V, dtype, seed=2)
    x[0, 100:] = fill
    x[1, :19990] = fill
    x[2, 4096:8192] = fill
    x[3, 8192:16384] = fill
    x[4] = fill
    x[5, :7000], x[5, 7001:] = fill, fill
    ids = _ids(T, V, 2)
    ids[0], ids[1], ids[4], ids[5] = [99, 100], [19990, 5], [0, 19999], [7000, 0]
    _check(x, ids, 12)
    lp, e, _, tl = _run(x, ids, 3)
    assert np.isfinite(lp).all() and np.isfinite(e).all() and np.isfinite(tl).all()
    assert lp[5, 0] == 0.0 and e[5] == 0.0 and abs(e[4] - np.log(V)) < 1e-5
    # mixed with tokens that cannot be drawn at all, and with whole chunks of those
    x[0, 200:], x[2, 8192:16384], x[4, ::2] = float("-inf"), float("-inf"), float("-inf")
    _check(x, ids, 12)
