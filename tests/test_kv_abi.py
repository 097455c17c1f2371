"""The entry points of include/qkv.h: every declared symbol is exported and
bound, bad arguments are refused on the host before anything is enqueued, and
the host-only frequency table follows its definition (CPU only: every other
call here ends in validation)."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest

import test_abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qkv.h")


@pytest.fixture(scope="module")
def q():
    return test_abi._lib()


def declared():
    return sorted(set(re.findall(r"QMM_API\s+[\w\s\*]+?\b(qkv_\w+)\s*\(", open(HEADER).read())))


def test_declared_exported_and_bound(q):
    from dequant_matmul_amd import kv
    out = subprocess.run(["nm", "-D", "--defined-only", test_abi.LIB], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert {s for s in exported if s.startswith("qkv_")} == set(declared()) == set(kv.SIGNATURES)


def test_structs_have_the_sizes_of_the_header(q, tmp_path):
    from dequant_matmul_amd import kv
    src = tmp_path / "s.c"
    src.write_text('#include "%s"\n#include <stdio.h>\nint main(void){printf("%%zu %%zu %%zu %%zu\\n",'
                   "sizeof(qkv_cache),sizeof(qkv_attn),sizeof(qkv_rope_scaling),"
                   "(size_t)&((qkv_attn*)0)->scale);return 0;}\n" % HEADER)
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(kv.CacheStruct), ctypes.sizeof(kv.AttnStruct), ctypes.sizeof(kv.RopeScaling),
                   kv.AttnStruct.scale.offset]


# ---------------------------------------------------------------- frequencies --

def test_plain_and_scaled_frequencies(q):
    i = np.arange(32)
    f, m = q.rope_freqs(64, 10000.0)
    plain = 10000.0 ** (-2 * i / 64)
    assert m == 1 and np.allclose(f.numpy(), plain, rtol=1e-15, atol=0)
    f, m = q.rope_freqs(64, 10000.0, "linear", factor=4)
    assert m == 1 and np.allclose(f.numpy(), plain / 4, rtol=1e-15, atol=0)
    f, _ = q.rope_freqs(64, 10000.0, "ntk", factor=4)
    assert np.allclose(f.numpy(), (10000.0 * 4 ** (64 / 62)) ** (-2 * i / 64), rtol=1e-14, atol=0)
    assert f[0] == 1 and abs(f[-1] - plain[-1] / 4) < 1e-15      # the slowest pair turns exactly `factor` times slower
    f, _ = q.rope_freqs(64, 10000.0, divisors=1.0 + i)
    assert np.allclose(f.numpy(), plain / (1 + i), rtol=1e-15, atol=0)
    f, m = q.rope_freqs(64, 10000.0, magnitude=1.5)
    assert m == 1.5 and np.allclose(f.numpy(), plain, rtol=1e-15, atol=0)
    f, _ = q.rope_freqs(2, 10000.0, "ntk", factor=4)
    assert f.tolist() == [1.0]


def test_yarn_frequencies(q):
    rot, base, s, trained = 128, 10000.0, 16.0, 4096.0
    f, m = q.rope_freqs(rot, base, "yarn", factor=s, trained=trained)
    plain = base ** (-2 * np.arange(64) / rot)
    turns = trained * plain / (2 * math.pi)
    assert m == pytest.approx(0.1 * math.log(16) + 1, rel=1e-15)
    share = f.numpy() / plain                          # 1 kept, 1/16 scaled
    assert np.allclose(share[turns > 33], 1, rtol=1e-15) and np.allclose(share[turns < 0.9], 1 / s, rtol=1e-15)
    assert np.all(np.diff(share) <= 1e-15)
    # a straight ramp over the pair index between
    mid = np.where((share < 0.999) & (share > 1 / s + 1e-3))[0]
    assert len(mid) > 5 and np.ptp(np.diff(share[mid])) < 1e-12
    assert q.rope_freqs(rot, base, "yarn", factor=0.5, trained=trained)[1] == 1


def test_band_frequencies(q):
    rot, base = 128, 500000.0
    f, m = q.rope_freqs(rot, base, "bands", factor=8.0, trained=8192)
    plain = base ** (-2 * np.arange(64) / rot)
    wave = 2 * math.pi / plain
    want = np.where(wave < 8192 / 4, plain, np.where(wave > 8192, plain / 8, 0))
    s = (8192 / wave - 1) / 3
    want = np.where(want == 0, (1 - s) * plain / 8 + s * plain, want)
    assert m == 1 and np.allclose(f.numpy(), want, rtol=1e-14, atol=0)


def test_frequency_refusals(q):
    for kw in (dict(rot=3), dict(rot=0), dict(rot=64, base=0.0), dict(rot=64, base=float("nan")),
               dict(rot=64, scaling="other"), dict(rot=64, scaling="linear", factor=0.0),
               dict(rot=64, scaling="linear", factor=float("inf")), dict(rot=64, scaling="yarn", factor=4.0),
               dict(rot=64, scaling="bands", factor=4.0, trained=8192, beta_fast=1.0),
               dict(rot=64, scaling="yarn", factor=4.0, trained=4096, base=0.5),
               dict(rot=64, divisors=[0.0] * 32), dict(rot=64, divisors=[1.0] * 31), dict(rot=65540),
               dict(rot=64, magnitude=float("nan"))):
        with pytest.raises((ValueError, q.QmmError)):
            q.rope_freqs(**kw)


# ------------------------------------------------------------------- refusals --
# Addresses that are never dereferenced.
A = 1 << 20
MIS = A + 4


def cache(q, **kw):
    from dequant_matmul_amd import kv
    d = dict(k=A, v=A, pages=4, type=q.Q8_0, kv_heads=2, head_dim=64, page_size=64)
    d.update(kw)
    return kv.CacheStruct(*[d[n] for n, _ in kv.CacheStruct._fields_])


BAD_CACHES = [(dict(type=7), "ERR_TYPE"), (dict(type=2), "ERR_TYPE"), (dict(kv_heads=0), "ERR_SHAPE"),
              (dict(kv_heads=1025), "ERR_SHAPE"), (dict(head_dim=60), "ERR_SHAPE"), (dict(head_dim=0), "ERR_SHAPE"),
              (dict(head_dim=264), "ERR_SHAPE"), (dict(page_size=32), "ERR_SHAPE"), (dict(page_size=96), "ERR_SHAPE"),
              (dict(page_size=0), "ERR_SHAPE"), (dict(page_size=-64), "ERR_SHAPE"), (dict(pages=-1), "ERR_SHAPE"),
              (dict(pages=1 << 25), "ERR_SHAPE"), (dict(k=None), "ERR_NULL"), (dict(v=None), "ERR_NULL"),
              (dict(k=MIS), "ERR_ALIGN"), (dict(v=MIS), "ERR_ALIGN")]


def test_page_bytes(q):
    L = q.lib
    assert L.qkv_page_bytes(q.Q8_0, 8, 128, 64) == 8 * 64 * 136
    assert L.qkv_page_bytes(q.Q4_0, 8, 128, 128) == 8 * 128 * 72
    assert L.qkv_page_bytes(q.F16, 4, 64, 64) == 4 * 64 * 128
    assert L.qkv_page_bytes(q.F16, 32, 80, 64) == 32 * 64 * 192          # 80 dims in three blocks of 32
    assert L.qkv_page_bytes(q.Q8_0, 1, 8, 64) == 64 * 68 and L.qkv_page_bytes(q.Q8_0, 1, 136, 64) == 64 * 272
    for a in ((2, 8, 128, 64), (q.Q8_0, 0, 128, 64), (q.Q8_0, 8, 12, 64), (q.Q8_0, 8, 128, 48), (q.Q8_0, 8, 128, 16)):
        assert L.qkv_page_bytes(*a) == 0


def test_bad_caches_are_refused_everywhere(q):
    from dequant_matmul_amd import kv
    L = q.lib
    a = attn(q)
    for kw, err in BAD_CACHES:
        c = cache(q, **kw)
        p = ctypes.addressof(c)
        want = getattr(q, err)
        assert L.qkv_append(p, 0, A, 128, A, 128, 4, A, None, 0, 0, None) == want, kw
        assert L.qkv_read(p, 0, A, 4, A, A, None) == want, kw
        assert L.qkv_move(p, A, A, 1, 4, None) == want, kw
        assert L.qkv_attention(p, ctypes.addressof(a), None) == want, kw
        if err not in ("ERR_NULL", "ERR_ALIGN"):
            assert L.qkv_attn_workspace(p, ctypes.addressof(a)) == -1
    assert L.qkv_append(None, 0, A, 128, A, 128, 4, A, None, 0, 0, None) == q.ERR_NULL
    assert L.qkv_attention(None, ctypes.addressof(a), None) == q.ERR_NULL


def test_rope_refusals(q):
    L = q.lib
    ok = dict(dtype=0, x=A, stride=256, tokens=4, heads=2, dim=128, cs=A, pairs=64, inter=0, out=A, ostride=256, stream=None)

    def call(**kw):
        return L.qkv_rope(*{**ok, **kw}.values())
    assert call(dtype=2) == q.ERR_TYPE and call(dtype=-1) == q.ERR_TYPE
    for kw in (dict(tokens=-1), dict(heads=-1), dict(dim=-8), dict(dim=100), dict(pairs=65), dict(pairs=-1),
               dict(stride=255), dict(ostride=128), dict(stride=260, ostride=260, dim=132), dict(stride=512),
               dict(heads=1 << 17), dict(tokens=1 << 31)):
        assert call(**kw) == q.ERR_SHAPE, kw
    for kw in (dict(x=None), dict(out=None), dict(cs=None)):
        assert call(**kw) == q.ERR_NULL, kw
    for kw in (dict(x=MIS), dict(out=MIS), dict(cs=MIS), dict(stride=258, ostride=258),
               dict(dtype=1, stride=260, ostride=260)):
        assert call(**kw) == q.ERR_ALIGN, kw
    for kw in (dict(tokens=0, x=None), dict(heads=0, x=None), dict(dim=0, pairs=0, x=None)):
        assert call(**kw) == q.OK, kw
    P = lambda *a: L.qkv_rope_angles(*a, None)  # noqa: E731
    assert P(A, -1, A, 4, 1.0, A) == q.ERR_SHAPE and P(A, 1, A, -1, 1.0, A) == q.ERR_SHAPE
    assert P(A, 1, A, 4, float("nan"), A) == q.ERR_SHAPE and P(A, 1 << 31, A, 4, 1.0, A) == q.ERR_SHAPE
    assert P(None, 1, A, 4, 1.0, A) == P(A, 1, None, 4, 1.0, A) == P(A, 1, A, 4, 1.0, None) == q.ERR_NULL
    assert P(A + 2, 1, A, 4, 1.0, A) == P(A, 1, MIS, 4, 1.0, A) == P(A, 1, A, 4, 1.0, MIS) == q.ERR_ALIGN
    assert P(None, 0, None, 4, 1.0, None) == P(None, 4, None, 0, 1.0, None) == q.OK


def test_cache_call_refusals(q):
    L = q.lib
    c = cache(q)
    p = ctypes.addressof(c)
    ok = dict(c=p, dtype=0, k=A, ks=128, v=A, vs=128, tokens=4, slots=A, cs=None, pairs=0, inter=0, stream=None)

    def append(**kw):
        return L.qkv_append(*{**ok, **kw}.values())
    assert append(dtype=3) == q.ERR_TYPE
    for kw in (dict(tokens=-1), dict(ks=127), dict(vs=64), dict(pairs=33), dict(pairs=-1), dict(tokens=1 << 31)):
        assert append(**kw) == q.ERR_SHAPE, kw
    for kw in (dict(k=None), dict(v=None), dict(slots=None)):
        assert append(**kw) == q.ERR_NULL, kw
    for kw in (dict(k=MIS), dict(v=MIS), dict(slots=A + 1), dict(cs=MIS, pairs=32), dict(ks=130)):
        assert append(**kw) == q.ERR_ALIGN, kw
    assert append(tokens=0, k=None, v=None, slots=None) == q.OK
    assert L.qkv_read(p, 5, A, 4, A, A, None) == q.ERR_TYPE
    assert L.qkv_read(p, 0, A, -4, A, A, None) == q.ERR_SHAPE
    assert L.qkv_read(p, 0, None, 4, A, A, None) == q.ERR_NULL
    assert L.qkv_read(p, 0, A, 4, MIS, A, None) == L.qkv_read(p, 0, A + 2, 4, A, A, None) == q.ERR_ALIGN
    assert L.qkv_read(p, 0, A, 4, None, None, None) == L.qkv_read(p, 0, None, 0, A, A, None) == q.OK
    assert L.qkv_move(p, A, A, 1, 65, None) == L.qkv_move(p, A, A, -1, 4, None) == L.qkv_move(p, A, A, 1, -1, None) == q.ERR_SHAPE
    assert L.qkv_move(p, None, A, 1, 4, None) == L.qkv_move(p, A, None, 1, 4, None) == q.ERR_NULL
    assert L.qkv_move(p, A + 1, A, 1, 4, None) == q.ERR_ALIGN
    assert L.qkv_move(p, None, None, 0, 4, None) == L.qkv_move(p, None, None, 4, 0, None) == q.OK


def attn(_q, **kw):
    from dequant_matmul_amd import kv
    d = dict(q=A, out=A, q_stride=512, out_stride=512, tokens=4, batch=4, table=A, columns=3, ctx=A, qstart=None,
             mask=None, mask_words=0, max_q=1, max_ctx=190, workspace=A, workspace_bytes=1 << 30, heads=8, dtype=0,
             scale=0.125, reserved=0)
    d.update(kw)
    return kv.AttnStruct(*[d[n] for n, _ in kv.AttnStruct._fields_])


def test_attention_refusals(q):
    L = q.lib
    c = cache(q)
    p = ctypes.addressof(c)

    def call(**kw):
        a = attn(q, **kw)
        return L.qkv_attention(p, ctypes.addressof(a), None)
    assert L.qkv_attention(p, None, None) == q.ERR_NULL
    assert call(dtype=2) == q.ERR_TYPE
    for kw in (dict(tokens=-1), dict(batch=-1), dict(columns=-1), dict(mask_words=-1), dict(max_q=-1), dict(max_ctx=-1),
               dict(heads=0), dict(heads=7), dict(batch=65536, tokens=65536), dict(max_ctx=(1 << 31) - 1),
               dict(tokens=1 << 30), dict(tokens=5), dict(scale=float("nan")), dict(scale=float("-inf")),
               dict(q_stride=511), dict(out_stride=256)):
        assert call(**kw) == q.ERR_SHAPE, kw
    for kw in (dict(q=None), dict(out=None), dict(ctx=None), dict(table=None)):
        assert call(**kw) == q.ERR_NULL, kw
    for kw in (dict(q=MIS), dict(out=MIS), dict(ctx=A + 2), dict(table=A + 2), dict(qstart=A + 1),
               dict(mask=MIS, mask_words=1), dict(workspace=MIS), dict(q_stride=514)):
        assert call(**kw) == q.ERR_ALIGN, kw
    big = dict(max_ctx=100000, columns=2000)
    need = L.qkv_attn_workspace(p, ctypes.addressof(attn(q, **big)))
    assert need > 0
    assert call(workspace_bytes=need - 1, **big) == q.ERR_WORKSPACE
    assert call(workspace=None, **big) == q.ERR_NULL
    for kw in (dict(tokens=0, q=None), dict(batch=0, ctx=None), dict(max_q=0, out=None)):
        assert call(**kw) == q.OK, kw
    assert "workspace" in q.status_str(q.ERR_WORKSPACE)


def test_workspace_depends_on_sizes_alone(q):
    L = q.lib
    c = cache(q, k=None, v=None)
    p = ctypes.addressof(c)
    a = attn(q, q=None, out=None, table=None, ctx=None, workspace=None, workspace_bytes=0)
    assert L.qkv_attn_workspace(p, ctypes.addressof(a)) >= 0
    assert L.qkv_attn_workspace(p, ctypes.addressof(attn(q, heads=7))) == -1
    # one tile of context needs no split
    assert L.qkv_attn_workspace(p, ctypes.addressof(attn(q, max_ctx=64))) == 0
