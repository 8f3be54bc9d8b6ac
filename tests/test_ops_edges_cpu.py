"""Arguments of the entry points around the step that no other CPU test refuses."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def B():
    from sparse_attention_indexer_tcgen05_gb300 import build
    build.build()
    from sparse_attention_indexer_tcgen05_gb300 import binding
    return binding


@pytest.mark.parametrize("stochastic,status", [(0, 0), (1, 0), (2, 1), (-1, 1)])
def test_adamw_rounding_refused(B, stochastic, status):
    p = B.csa_adamw_params(step=1, beta1=0.9, beta2=0.99, stochastic=stochastic, seed=2 ** 64 - 1)
    assert B._lib.csa_adamw(ctypes.byref(p), None, 0, None) == status
