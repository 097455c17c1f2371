"""Sizes at the ends of their types at the entry points of include/qkv.h (CPU only:
every call ends in validation)."""
import ctypes

import pytest

import test_kv_abi as K
from test_kv_abi import A, q  # noqa: F401  (q: the fixture)


@pytest.mark.parametrize("pairs", [1 << 62, (1 << 62) + 1, (1 << 63) - 1])
def test_pairs_whose_double_wraps(q, pairs):  # noqa: F811
    assert q.lib.qkv_rope(0, A, 256, 4, 2, 128, A, pairs, 0, A, 256, None) == q.ERR_SHAPE
    c = K.cache(q)
    assert q.lib.qkv_append(ctypes.addressof(c), 0, A, 128, A, 128, 4, A, A, pairs, 0, None) == q.ERR_SHAPE
