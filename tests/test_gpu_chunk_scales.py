"""Attention of chunks with factors of the scores at both ends of fp32; tolerances as in test_gpu_chunk.py."""
import numpy as np
import pytest
import torch

from test_gpu_attention import _bf16, _filled, _gen
from test_gpu_chunk import _check_chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_expert_gb300 as mx
    return mx


@pytest.mark.parametrize("scale", [2.3e38, 2.4e38, 3.4028234663852886e38])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("P,d", [(16, 64), (64, 128)])
def test_largest_scales(mx, scale, sign, P, d):
    """Keys and queries so small that the scores are ordinary numbers."""
    lens = [300, 70]
    c, table = _filled(mx, lens, P, 2, d, -(-300 // P), 3, spread=lambda rng, s: 40 + rng.integers(-2, 3, size=s))
    _check_chunk(mx, c, table, [40, 70], lens, 4, scale=sign * float(np.float32(scale)), q=_bf16(_gen(1), 110, 4, d, spread=2.0 ** -50))


@pytest.mark.parametrize("scale", [0.0, 1.4e-45, 1e-40, 1e-20])
def test_smallest_scales(mx, scale):
    lens = [300, 70]
    c, table = _filled(mx, lens, 32, 2, 64, 10, 4)
    _check_chunk(mx, c, table, [40, 70], lens, 4, scale=float(np.float32(scale)))
    _check_chunk(mx, c, table, [40, 70], lens, 4, scale=float(np.float32(scale)), q=_bf16(_gen(2), 110, 4, 64, spread=1e30))
