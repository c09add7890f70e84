"""The soft-CE against top logits at the ends of its arguments' ranges, against the fp64 oracle."""

import numpy as np
import pytest
import torch

from _serving import DEV, f64
from _top import logits
from oracle import top as ot
from speculative_decoding_draft_eagle_gb300 import ops
from test_soft_ce_topk_gpu import _check, _g, _teacher

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()
    yield
    assert ops.stt_device_error() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V,K", [(300, 7), (60001, 200)])
def test_a_teacher_row_without_logits(V, K, bf16):
    """Valid places with values of -inf, and the log-sum-exp of -inf that such a row has: none of
    them is an entry, and no other row notices."""
    N = 5
    val, idx = _teacher(N, V, K)
    val[1], val[3, ::2], val[4, 1:] = -np.inf, -np.inf, -np.inf
    lse = ot.logsumexp(val.astype(np.float64)).astype(np.float32)
    assert lse[1] == -np.inf
    got = _check(logits(N, V, bf16), val, idx, _g(N, masked=0), lse)
    assert not got[1].any()
    assert not _check(logits(N, V, bf16), val, idx, _g(N, masked=0), None, 2.0)[1].any()
