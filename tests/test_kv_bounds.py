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


def test_more_row_groups_than_a_launch_holds(q):  # noqa: F811
    """Row groups times kv heads past 65535 are refused, by the workspace query too."""
    c = K.cache(q, kv_heads=1024)
    for dtype in (0, 1):
        a = K.attn(q, tokens=1 << 17, batch=1, heads=1024, q_stride=1 << 16, out_stride=1 << 16, max_q=1 << 17,
                   dtype=dtype)
        assert q.lib.qkv_attn_workspace(ctypes.addressof(c), ctypes.addressof(a)) == -1
        assert q.lib.qkv_attention(ctypes.addressof(c), ctypes.addressof(a), None) == q.ERR_SHAPE


def test_fewer_sequences_may_need_more_workspace(q):  # noqa: F811
    """As the header says (256 compute units, also where there is no device)."""
    c = K.cache(q, kv_heads=8, head_dim=128)

    def call(b, **kw):
        return K.attn(q, tokens=b, batch=b, heads=32, q_stride=4096, out_stride=4096, max_q=1, max_ctx=32000,
                      columns=500, **kw)
    need = {b: q.lib.qkv_attn_workspace(ctypes.addressof(c), ctypes.addressof(call(b))) for b in (7, 16, 64)}
    assert need == {7: 1164800, 16: 1064960, 64: 0}
    a = call(7, workspace_bytes=need[16])
    assert q.lib.qkv_attention(ctypes.addressof(c), ctypes.addressof(a), None) == q.ERR_WORKSPACE


@pytest.mark.parametrize("trained,slow,share", [(4.0, 1.0, 1 / 16), (500.0, 100.0, 1 / 16), (1e30, 1.0, 1.0)])
def test_yarn_where_all_pairs_are_on_one_side(q, trained, slow, share):  # noqa: F811
    """Every pair below beta_slow turns of the trained context is scaled, the first one
    too; every pair above beta_fast is not."""
    f, _ = q.rope_freqs(64, 10000.0, "yarn", factor=16.0, trained=trained, beta_slow=slow, beta_fast=32 * slow)
    plain, _ = q.rope_freqs(64, 10000.0)
    turns = trained * plain / (2 * 3.141592653589793)
    assert (turns < slow).all() or (turns > 32 * slow).all()
    assert (abs(f / plain - share) < 1e-15).all()
