"""The K largest logits at the ends of what rows hold."""

import numpy as np
import pytest
import torch

from _serving import f64, gen
from _top import in_rows
from oracle import top as ot
from speculative_decoding_draft_eagle_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()
    yield
    assert ops.stt_device_error() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("N,V,K", [(3, 50, 20), (2, 151936, 100), (400, 9001, 30)])
@pytest.mark.parametrize("layout", ["dense", "odd"])
def test_zeros_keep_their_signs(N, V, K, bf16, layout):
    """Zeros of both signs count as equal, and are given as they are."""
    g = gen(V)
    z = -torch.rand(N, V, generator=g) - 0.5
    z[torch.rand(N, V, generator=g) < 3.0 * K / V] = 0.0
    z = torch.where((z == 0) & (torch.rand(N, V, generator=g) < 0.5), -0.0, z)
    z = z.to(torch.bfloat16 if bf16 else torch.float32)
    v, i, _ = ops.stt_top_logits(in_rows(z, layout), K)
    _, I, _ = ot.top(f64(z), K)
    assert np.array_equal(i.cpu().numpy(), I)
    want = np.take_along_axis(f64(z), I, 1)
    assert np.array_equal(f64(v), want) and np.array_equal(np.signbit(f64(v)), np.signbit(want))
    assert np.signbit(want[want == 0]).any() and not np.signbit(want[want == 0]).all()
