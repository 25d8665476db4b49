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
