"""Limits of the sizes that the entries of include/qst.h take (CPU only: every call
here ends in validation)."""
import ctypes

import pytest

import test_abi

A = 1 << 20          # never dereferenced


@pytest.fixture(scope="module")
def q():
    return test_abi._lib()


@pytest.fixture(scope="module")
def step(q):
    from dequant_matmul_amd import step
    return step


def lora_args(step, **kw):
    d = dict(x=A, adapter=A, workspace=A, workspace_bytes=1 << 60, x_stride=1 << 31, tokens=1, batch=1, k=64, adapters=1,
             rank=8, dtype=0, targets=1)
    d.update(kw)
    return step.LoraArgs(**d)


@pytest.mark.parametrize("k,good", [(8, True), (2 ** 31 - 2 ** 14, True), (2 ** 31 - 2 ** 14 + 8, False),
                                    (2 ** 31 - 8, False), (2 ** 31, False), (0, False), (12, False)])
def test_k_of_adapters(q, step, k, good):
    """No part of k ends past 2^31."""
    a = lora_args(step, k=k)
    assert (q.lib.qst_lora_workspace(ctypes.addressof(a)) > 0) == good
    if not good:
        t = step.LoraTarget(A, A, None, A, 8)
        assert q.lib.qst_lora(ctypes.addressof(a), ctypes.addressof(t), None) == q.ERR_SHAPE


def test_the_bound_of_the_workspace(q, step):
    """What the header gives as the most for any smaller call of a step, over sizes on
    either side of every rule; and that a smaller call can need more than a larger one."""
    def need(**kw):
        return q.lib.qst_lora_workspace(ctypes.addressof(lora_args(step, **kw)))
    for targets in (1, 3, 8):
        for rank in (8, 24, 64, 128, 256):
            for k in (8, 1024, 1032, 4096, 14336, 65544, 1 << 20):
                for tokens in (1, 2, 16, 53, 512, 3000, 8192, 100000):
                    bound = 4 * targets * tokens * rank * min(64, -(-k // 1024))
                    for batch in (1, 4, 16, 60, 200, 65535):
                        assert 0 < need(targets=targets, rank=rank, k=k, tokens=tokens, batch=batch) <= bound
    assert need(targets=3, rank=32, k=14336, tokens=3000, batch=1) > need(targets=3, rank=32, k=14336, tokens=8192, batch=4)


def test_calls_are_packed_as_the_structs(step):
    """The bytes that a call hands over lie where the structs' fields do."""
    for packer, struct in ((step._PLAN, step.PlanArgs), (step._NORM, step.NormArgs), (step._LORA, step.LoraArgs),
                           (step._PROBLEM, step.GemvProblem), (step._TARGET, step.LoraTarget)):
        values = [0.5 if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(struct._fields_)]
        s = struct.from_buffer_copy(packer.pack(*values))
        assert [getattr(s, name) for name, _ in struct._fields_] == values
