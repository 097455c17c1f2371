"""Every call of the binding reaches the library with its tensors' device current
and on torch's current stream of that device (CPU only: the library's functions,
torch's device functions and the tensors are stand-ins)."""
import pytest
import torch

import test_abi

F32, F16, I32, I64, F64, U8 = (torch.float32, torch.float16, torch.int32, torch.int64, torch.float64, torch.uint8)


class Fake:
    """A contiguous device tensor as far as the binding looks at one."""
    is_cuda = True

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", device)

    def stride(self):
        return tuple(self.shape[i + 1:].numel() for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 1 << 20


class Library:
    """Notes the current device and the stream (a call's last argument) of every
    function with one."""

    def __init__(self, real, state):
        self.real, self.state, self.calls = real, state, []

    def __getattr__(self, name):
        if name in ("qmm_row_bytes", "qkv_page_bytes", "qmm_status_str"):
            return getattr(self.real, name)

        def f(*args):
            self.calls.append((name, self.state["now"], args[-1]))
            return 0
        return f


@pytest.fixture
def seat(monkeypatch):
    """q, its kv module and a record of calls, device 0 current of several; the
    stream of device i is 100 + i."""
    q = test_abi._lib()
    from dequant_matmul_amd import kv
    state = {"now": 0, "entered": 0}

    class device:
        def __init__(self, d):
            self.d = d.index if isinstance(d, torch.device) else d

        def __enter__(self):
            self.before, state["now"] = state["now"], self.d
            state["entered"] += 1

        def __exit__(self, *a):
            state["now"] = self.before
    rec = Library(q.lib, state)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["now"])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: type("S", (), {"cuda_stream": 100 + d.index}))
    if hasattr(kv, "_raw_stream"):
        monkeypatch.setattr(kv, "_raw_stream", torch._C._cuda_getCurrentRawStream)
    monkeypatch.setattr(q, "lib", rec)
    monkeypatch.setattr(kv, "lib", rec)
    return q, rec, state


def calls(q, d):
    """name of the library's function -> a call of the binding with tensors on device d."""
    def t(dtype, *shape):
        return Fake(shape, dtype, d)
    cache = q.KVCache(q.Q8_0, 2, 64, 4, k=t(U8, 4 * 64 * 2 * 68), v=t(U8, 4 * 64 * 2 * 68))
    w = t(U8, 8 * q.row_bytes(q.Q8_0, 64))
    x, y = t(F32, 1, 64), t(F32, 1, 8)
    rows, kv = t(F32, 5, 4, 64), t(F32, 5, 2, 64)
    cs, slots = t(F32, 5, 32, 2), t(I32, 5)
    problem = [(w, q.Q8_0, 8, 64, x, y, 0)]
    return {
        "qkv_rope_angles": lambda: q.rope_angles(slots, t(F64, 32), out=cs),
        "qkv_rope": lambda: q.rope(rows, cs, out=rows),
        "qkv_append": lambda: q.kv_append(cache, kv, kv, slots, cs=cs),
        "qkv_read": lambda: q.kv_read(cache, slots, k_out=kv, v_out=kv),
        "qkv_move": lambda: q.kv_move(cache, t(I32, 1, 5), t(I32, 1, 5)),
        "qkv_attention": lambda: q.attention(cache, rows, t(I32, 1, 4), t(I32, 1), out=t(F32, 5, 4, 64),
                                             workspace=t(U8, 1 << 20)),
        "qmm_dequant": lambda: q.dequant(w, q.Q8_0, 8, 64, out=t(F32, 8, 64)),
        "qmm_dequant_f16": lambda: q.dequant_f16(w, q.Q8_0, 8, 64, out=t(F16, 8, 64)),
        "qmm_embed": lambda: q.embed(w, q.Q8_0, 8, 64, slots, out=t(F32, 5, 64)),
        "qmm_embed_f16": lambda: q.embed(w, q.Q8_0, 8, 64, slots, dtype=F16, out=t(F16, 5, 64)),
        "qmm_quantize": lambda: q.quantize(t(F32, 8, 64), q.Q8_0, out=t(U8, 8, 68)),
        "qmm_quantize_f16": lambda: q.quantize(t(F16, 8, 64), q.Q8_0, out=t(U8, 8, 68)),
        "qmm_gemv": lambda: q.gemv(w, q.Q8_0, 8, 64, x, out=y),
        "qmm_gemv_multi": lambda: q.gemv_multi([w], q.Q8_0, [8], 64, [x], outs=[y]),
        "qmm_gemv_pass": lambda: q.gemv_pass(problem),
        "qmm_gemm_prefill": lambda: q.gemm_prefill(w, q.Q8_0, 8, 64, t(F16, 5, 64), out=t(F32, 5, 8)),
    }


def test_every_call_runs_on_its_tensors_device(seat):
    q, rec, state = seat
    from dequant_matmul_amd import kv
    # every function of the library that takes a stream is called below
    streams = {n for n, (_, a) in {**q.SIGNATURES, **kv.SIGNATURES}.items()
               if n not in ("qmm_block_elems", "qmm_block_bytes", "qmm_row_bytes", "qmm_status_str", "qmm_version",
                            "qkv_rope_freqs", "qkv_page_bytes", "qkv_attn_workspace")}
    for d in (0, 1, 3):
        every = calls(q, d)
        assert set(every) == streams
        for name, call in every.items():
            del rec.calls[:]
            state["entered"] = 0
            call()
            assert rec.calls == [(name, d, 100 + d)], name
            assert state["now"] == 0 and state["entered"] == (d != 0), name     # and no guard where none is needed


def test_a_pass_on_a_stream_of_the_callers(seat):
    q, rec, state = seat
    w, x, y = Fake((8 * 68,), U8, 2), Fake((64,), F32, 2), Fake((8,), F32, 2)
    q.gemv_pass([(w, q.Q8_0, 8, 64, x, y, 0)], stream=7)
    assert rec.calls == [("qmm_gemv_pass", 2, 7)]
    q.gemv_pass([])
    q.gemv_multi([], q.Q8_0, [], 64, [])
    assert [c[0] for c in rec.calls] == ["qmm_gemv_pass", "qmm_gemv_pass", "qmm_gemv_multi"]


def test_the_workspace_is_that_of_the_caches_device(seat, monkeypatch):
    q, rec, state = seat
    cache = q.KVCache(q.Q8_0, 2, 64, 4, k=Fake((4 * 64 * 2 * 68,), U8, 1), v=Fake((4 * 64 * 2 * 68,), U8, 1))
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: (n, device))
    assert q.attention_workspace(cache, Fake((5, 4, 64), F32, 1), Fake((1, 4), I32, 1)) == (0, torch.device("cuda", 1))
    assert rec.calls[0][:2] == ("qkv_attn_workspace", 1)
