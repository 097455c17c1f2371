"""The entry points of include/qst.h: every declared symbol is exported and bound,
structs have the sizes of the header, and bad arguments are refused on the host
before anything is enqueued (CPU only: every call here ends in validation)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import test_abi
from test_devices import F16, F32, I32, U8, Fake, seat  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qst.h")
A = 1 << 20          # never dereferenced


@pytest.fixture(scope="module")
def q():
    return test_abi._lib()


@pytest.fixture(scope="module")
def step(q):
    from dequant_matmul_amd import step
    return step


def test_declared_exported_and_bound(q, step):
    declared = set(re.findall(r"QMM_API\s+[\w\s\*]+?\b(qst_\w+)\s*\(", open(HEADER).read()))
    out = subprocess.run(["nm", "-D", "--defined-only", test_abi.LIB], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert {s for s in exported if s.startswith("qst_")} == declared == set(step.SIGNATURES)


def test_structs_have_the_layout_of_the_header(step, tmp_path):
    pairs = [("qst_plan_args", step.PlanArgs), ("qst_norm_args", step.NormArgs), ("qst_gemv_problem", step.GemvProblem),
             ("qst_lora_target", step.LoraTarget), ("qst_lora_args", step.LoraArgs)]
    want = []
    code = '#include "%s"\n#include <stdio.h>\n#include <stddef.h>\nint main(void){\n' % HEADER
    for name, py in pairs:
        code += 'printf("%%zu\\n", sizeof(%s));\n' % name
        want.append(ctypes.sizeof(py))
        for field, _ in py._fields_:
            code += 'printf("%%zu\\n", offsetof(%s, %s));\n' % (name, field)
            want.append(getattr(py, field).offset)
    src = tmp_path / "s.c"
    src.write_text(code + "return QST_Q8_0 == %d ? 0 : 1;}\n" % step._OUT_Q8)
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == want
    # ... and so have the bytes that calls are made of
    for packed, py in ((step._PLAN, step.PlanArgs), (step._NORM, step.NormArgs), (step._PROBLEM, step.GemvProblem),
                       (step._TARGET, step.LoraTarget), (step._LORA, step.LoraArgs)):
        values = list(range(1, len(py._fields_) + 1))
        assert packed.pack(*values) == bytes(py(*values))


def struct(cls, d, **kw):
    assert set(kw) <= set(d)
    d = {**d, **kw}
    return cls(*[d[n] for n, _ in cls._fields_])


def test_plan_refusals(q, step):
    ok = dict(table=A, ctx=A, fresh=None, free=A, count=A, qstart=A, slots=A, pos=A, granted=A, left=A, batch=3,
              columns=4, pages=100, page_size=64, tokens=9)

    def call(**kw):
        a = struct(step.PlanArgs, ok, **kw)
        return q.lib.qst_plan(ctypes.addressof(a), None)
    assert q.lib.qst_plan(None, None) == q.ERR_NULL
    for kw in (dict(batch=-1), dict(batch=65536), dict(columns=-1), dict(columns=1 << 31), dict(pages=-1),
               dict(pages=1 << 25), dict(page_size=32), dict(page_size=96), dict(page_size=0), dict(page_size=1 << 31),
               dict(tokens=-1), dict(tokens=1 << 31)):
        assert call(**kw) == q.ERR_SHAPE, kw
    for name in ("table", "ctx", "free", "count", "qstart", "slots", "pos", "granted", "left"):
        assert call(**{name: None}) == q.ERR_NULL, name
    for name in ("table", "ctx", "fresh", "free", "count", "qstart", "slots", "pos", "granted", "left"):
        assert call(**{name: A + 2}) == q.ERR_ALIGN, name


def test_trim_refusals(q):
    ok = dict(table=A, batch=3, columns=4, held=A, kept=A, free=A, count=A, pages=100, page=64, left=A, stream=None)

    def call(**kw):
        return q.lib.qst_trim(*{**ok, **kw}.values())
    for kw in (dict(batch=-1), dict(batch=65536), dict(columns=-1), dict(columns=1 << 31), dict(pages=-1),
               dict(pages=1 << 25), dict(page=63)):
        assert call(**kw) == q.ERR_SHAPE, kw
    for name in ("table", "held", "kept", "free", "count", "left"):
        assert call(**{name: None}) == q.ERR_NULL, name
        assert call(**{name: A + 1}) == q.ERR_ALIGN, name


def test_norm_refusals(q, step):
    ok = dict(x=A, residual=2 * A, sum=3 * A, weight=A, out=4 * A, x_stride=64, residual_stride=64, sum_stride=64,
              out_stride=64, tokens=3, heads=1, dim=64, eps=1e-5, x_type=0, residual_type=0, out_type=0)

    def call(**kw):
        a = struct(step.NormArgs, ok, **kw)
        return q.lib.qst_norm(ctypes.addressof(a), None)
    assert q.lib.qst_norm(None, None) == q.ERR_NULL
    for kw in (dict(x_type=2), dict(x_type=-1), dict(residual_type=2), dict(out_type=2), dict(out_type=16)):
        assert call(**kw) == q.ERR_TYPE, kw
    for kw in (dict(tokens=-1), dict(tokens=1 << 31), dict(heads=-1), dict(heads=65536), dict(dim=-1), dict(dim=65537),
               dict(eps=0.0), dict(eps=-1e-5), dict(eps=float("nan")), dict(eps=float("inf")), dict(x_stride=63),
               dict(residual_stride=0), dict(sum_stride=63), dict(out_stride=63), dict(heads=2), dict(x_stride=1 << 41),
               dict(out_type=step._OUT_Q8, dim=40),
               # one buffer under two strides or types, the norm in the sum's place
               dict(sum=A, x_stride=128), dict(sum=2 * A, sum_stride=72), dict(sum=2 * A, out=2 * A), dict(sum=4 * A),
               dict(out=A, x_type=1), dict(out=A, x_stride=80), dict(out=2 * A, residual_type=1),
               dict(out=2 * A, out_stride=72), dict(sum=A, x_type=1),
               dict(out=A, out_type=step._OUT_Q8), dict(out=2 * A, out_type=step._OUT_Q8)):
        assert call(**kw) == q.ERR_SHAPE, kw
    for kw in (dict(x=None), dict(out=None), dict(out=None, out_type=step._OUT_Q8)):
        assert call(**kw) == q.ERR_NULL, kw
    for kw in (dict(x=A + 2), dict(x=A + 1, x_type=1), dict(residual=A + 2), dict(sum=A + 2), dict(out=A + 2),
               dict(weight=A + 2), dict(out=A + 8, out_type=step._OUT_Q8)):
        assert call(**kw) == q.ERR_ALIGN, kw
    for kw in (dict(tokens=0, x=None), dict(heads=0, x=None), dict(dim=0, x=None)):
        assert call(**kw) == q.OK, kw


def test_gemv_q8_refusals(q, step):
    def call(*probs, k=256, x=A, batch=1):
        t = (step.GemvProblem * max(1, len(probs)))()
        for i, p in enumerate(probs):
            t[i] = struct(step.GemvProblem, dict(w=A, y=A, n=4, type=q.Q4_K, reserved=0), **p)
        return q.lib.qst_gemv_q8(len(probs), ctypes.addressof(t), k, x, batch, None)
    assert q.lib.qst_gemv_q8(-1, None, 256, A, 1, None) == q.ERR_SHAPE
    assert q.lib.qst_gemv_q8(0, None, 256, A, 1, None) == q.OK
    assert q.lib.qst_gemv_q8(1, None, 256, A, 1, None) == q.ERR_NULL
    assert call(dict(type=6)) == call(dict(type=-1)) == q.ERR_TYPE
    assert call({}, k=48) == call({}, k=128) == call({}, k=-256) == call({}, k=1 << 31) == q.ERR_SHAPE
    assert call({}, batch=9) == call({}, batch=-1) == call(dict(n=-1)) == call(dict(n=1 << 31)) == q.ERR_SHAPE
    assert call({}, dict(type=q.Q8_0), k=32) == q.ERR_SHAPE          # k of one problem is no multiple of its blocks
    assert call(dict(w=None)) == call(dict(y=None)) == call({}, x=None) == q.ERR_NULL
    assert call(dict(w=A + 8)) == call(dict(y=A + 4)) == call({}, x=A + 2) == q.ERR_ALIGN
    assert call({}, dict(w=None)) == q.ERR_NULL                      # nothing of the first is enqueued either
    assert call(dict(n=0, w=None, y=None), x=None) == call({}, batch=0, x=None) == q.OK


def lora_args(step, **kw):
    return struct(step.LoraArgs, dict(x=A, adapter=A, qstart=None, scale=None, ranks=None, workspace=A,
                                      workspace_bytes=1 << 40, x_stride=64, tokens=6, batch=3, k=64, adapters=2, rank=16,
                                      dtype=0, targets=2), **kw)


def test_lora_refusals(q, step):
    def call(t=({}, {}), **kw):
        tab = (step.LoraTarget * 9)()
        for i in range(9):
            tab[i] = struct(step.LoraTarget, dict(a=A, b=A, base=None, y=A, n=5), **(t[i] if i < len(t) else {}))
        a = lora_args(step, **kw)
        return q.lib.qst_lora(ctypes.addressof(a), ctypes.addressof(tab), None)
    assert q.lib.qst_lora(None, None, None) == q.ERR_NULL
    assert q.lib.qst_lora(ctypes.addressof(lora_args(step)), None, None) == q.ERR_NULL
    assert call(dtype=2) == q.ERR_TYPE
    for kw in (dict(tokens=-1), dict(tokens=1 << 31), dict(batch=-1), dict(batch=65536), dict(k=0), dict(k=60),
               dict(k=1 << 31), dict(adapters=-1), dict(rank=0), dict(rank=12), dict(rank=264), dict(targets=-1),
               dict(targets=9), dict(tokens=7), dict(x_stride=60), dict(t=[dict(n=-1)]), dict(t=[dict(n=(1 << 24) + 1)]),
               dict(tokens=1 << 20, batch=1 << 10)):
        assert call(**kw) == q.ERR_SHAPE, kw
    for kw in (dict(x=None), dict(adapter=None), dict(workspace=None), dict(t=[dict(a=None)]), dict(t=[{}, dict(b=None)]),
               dict(t=[dict(y=None)])):
        assert call(**kw) == q.ERR_NULL, kw
    for kw in (dict(x=A + 8), dict(adapter=A + 2), dict(qstart=A + 2), dict(scale=A + 2), dict(ranks=A + 1),
               dict(workspace=A + 4), dict(x_stride=66), dict(dtype=1, x_stride=68), dict(t=[dict(a=A + 8)]),
               dict(t=[dict(b=A + 2)]), dict(t=[dict(y=A + 4)]), dict(t=[dict(base=A + 8)])):
        assert call(**kw) == q.ERR_ALIGN, kw
    need = q.lib.qst_lora_workspace(ctypes.addressof(lora_args(step)))
    assert need > 0 and call(workspace_bytes=need - 1) == q.ERR_WORKSPACE
    for kw in (dict(tokens=0, x=None), dict(batch=0, adapter=None), dict(targets=0), dict(t=[dict(n=0, y=None)] * 2)):
        assert call(**kw) == q.OK, kw


def test_lora_workspace_looks_at_sizes_alone(q, step):
    a = lora_args(step, x=None, adapter=None, workspace=None, workspace_bytes=0)
    assert q.lib.qst_lora_workspace(ctypes.addressof(a)) > 0
    assert q.lib.qst_lora_workspace(ctypes.addressof(lora_args(step, rank=4))) == -1
    assert q.lib.qst_lora_workspace(None) == -1
    for kw in (dict(targets=0), dict(tokens=0), dict(batch=0), dict(adapters=0)):
        assert q.lib.qst_lora_workspace(ctypes.addressof(lora_args(step, **kw))) >= 0


# ---------------------------------------------------------------- the binding --

def calls(q, d):
    def t(dtype, *shape):
        return Fake(shape, dtype, d)
    table, free, count, i3 = t(I32, 3, 4), t(I32, 50), t(I32, 1), t(I32, 3)
    w, x8 = t(U8, 8 * q.row_bytes(q.Q8_0, 64)), t(U8, 2, 68)
    x = Fake((6, 64), F32, d)
    x.stride = lambda i=None: (64, 1) if i is None else (64, 1)[i]
    target = [(t(F16, 2, 16, 64), t(F16, 2, 5, 16), t(F32, 6, 5))]
    return {
        "qst_plan": lambda: q.kv_plan(table, i3, i3, free, count, 9, out=(t(I32, 4), t(I32, 9), t(I32, 9), i3, count)),
        "qst_trim": lambda: q.kv_trim(table, i3, i3, free, count, left=count),
        "qst_norm": lambda: q.rms_norm(t(F32, 3, 64), t(F32, 64), residual=t(F32, 3, 64), sum_out=t(F32, 3, 64),
                                       out=t(F32, 3, 64)),
        "qst_gemv_q8": lambda: q.gemv_q8(w, q.Q8_0, 8, 64, x8, out=t(F32, 2, 8)),
        "qst_lora": lambda: q.lora(x, target, i3, workspace=t(U8, 1 << 20)),
    }


def test_every_call_runs_on_its_tensors_device(seat, step, monkeypatch):  # noqa: F811
    q, rec, state = seat
    monkeypatch.setattr(step, "lib", rec)
    for d in (0, 1, 3):
        every = calls(q, d)
        assert set(every) == set(step.SIGNATURES) - {"qst_lora_workspace"}
        for name, call in every.items():
            del rec.calls[:]
            call()
            assert rec.calls == [(name, d, 100 + d)], name
            assert state["now"] == 0


def test_the_binding_refuses(seat, step, monkeypatch):  # noqa: F811
    q, rec, _ = seat
    monkeypatch.setattr(step, "lib", rec)

    def t(dtype, *shape, d=0):
        return Fake(shape, dtype, d)
    i3, table, free, count = t(I32, 3), t(I32, 3, 4), t(I32, 50), t(I32, 1)
    x, w8, x8 = t(F32, 3, 64), t(U8, 8 * 68), t(U8, 2, 68)
    a, b, y = t(F16, 2, 16, 64), t(F16, 2, 5, 16), t(F32, 6, 5)
    xl = Fake((6, 64), F32, 0)
    xl.stride = lambda i=None: (64, 1) if i is None else (64, 1)[i]
    bad = [
        lambda: q.kv_plan(table, t(I32, 2), None, free, count, 9), lambda: q.kv_plan(table, i3, t(F32, 3), free, count, 9),
        lambda: q.kv_plan(table, i3, None, free, t(I32, 2), 9), lambda: q.kv_plan(t(I32, 12), i3, None, free, count, 9),
        lambda: q.kv_plan(table, t(I32, 3, d=1), None, free, count, 9),
        lambda: q.kv_plan(table, i3, None, free, count, 9, out=(t(I32, 4), t(I32, 8), t(I32, 9), i3, count)),
        lambda: q.kv_trim(table, i3, t(I32, 4), free, count), lambda: q.kv_trim(table, i3, i3, free, count, left=i3),
        lambda: q.rms_norm(t(U8, 3, 64)), lambda: q.rms_norm(t(F32, 64)), lambda: q.rms_norm(x, t(F16, 64)),
        lambda: q.rms_norm(x, t(F32, 32)), lambda: q.rms_norm(x, residual=t(F32, 3, 32)),
        lambda: q.rms_norm(x, residual=t(F32, 3, 64), sum_out=t(F16, 3, 64)),
        lambda: q.rms_norm(x, qtype=q.Q4_0), lambda: q.rms_norm(x, qtype=q.Q8_0, dtype=F16),
        lambda: q.rms_norm(t(F32, 3, 40), qtype=q.Q8_0), lambda: q.rms_norm(x, out=t(F16, 3, 64), dtype=F32),
        lambda: q.rms_norm(x, residual=t(F32, 3, 64, d=1)),
        lambda: q.gemv_q8(w8, q.Q8_0, 8, 64, t(U8, 2, 64)), lambda: q.gemv_q8(w8, q.Q8_0, 8, 64, t(F32, 2, 68)),
        lambda: q.gemv_q8(w8, q.Q8_0, 9, 64, x8), lambda: q.gemv_q8(t(U8, 8 * 68, d=1), q.Q8_0, 8, 64, x8),
        lambda: q.gemv_q8_multi([w8], [q.Q8_0, q.Q8_0], [8], 64, x8),
        lambda: q.gemv_q8(w8, q.Q8_0, 8, 64, x8, out=t(F32, 2, 9)),
        lambda: q.lora(xl, [(a, t(F16, 2, 5, 8), y)], i3), lambda: q.lora(xl, [(t(F32, 2, 16, 64), b, y)], i3),
        lambda: q.lora(xl, [(a, b, t(F32, 5, 5))], i3), lambda: q.lora(xl, [(a, b, y, t(F32, 6, 4))], i3),
        lambda: q.lora(xl, [(a, b, y)], i3, qstart=i3), lambda: q.lora(xl, [(a, b, y)], i3, scale=t(F32, 3)),
        lambda: q.lora(xl, [(a, b, y)], i3, ranks=t(F32, 2)), lambda: q.lora(xl, [(a, b, y)], t(I32, 3, 1)),
        lambda: q.lora(xl, [(a, b, y)], i3, workspace=t(F32, 9)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
        assert not [c for c in rec.calls if not c[0].endswith("workspace")], i
    assert torch is not None
