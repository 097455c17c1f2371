"""A call reports its own launch: an error that an earlier, unrelated call of the
host thread has left (here a device ordinal that does not exist, refused by the
runtime on the host) is neither reported by it nor taken away."""
import ctypes

import pytest

import qmm_inputs as G

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_matmul_amd as q  # noqa: E402

DEV = "cuda:0"


@pytest.fixture
def hip():
    """The HIP runtime that torch has loaded; no error is left behind."""
    paths = {line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line}
    assert len(paths) == 1
    h = ctypes.CDLL(paths.pop())
    yield h
    h.hipGetLastError()


def every():
    def i32(*v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)
    cache = q.KVCache(q.Q8_0, 2, 64, 4)
    cache.k.zero_()
    cache.v.zero_()
    n, k = 32, 256
    w = torch.zeros(n * q.row_bytes(G.Q4_K, k), dtype=torch.uint8, device=DEV)
    w8 = torch.zeros(n * q.row_bytes(G.Q8_0, k), dtype=torch.uint8, device=DEV)
    x, y = torch.zeros(2, k, device=DEV), torch.full((2, n), 7.0, device=DEV)
    x1, y1 = x[:1], torch.full((1, n), 7.0, device=DEV)
    rows, kv, out = (torch.zeros(3, h, 64, device=DEV) for h in (8, 2, 8))
    many, more = torch.zeros(40, 8, 64, device=DEV), torch.zeros(40, 8, 64, device=DEV)
    src, dst = i32(0, 1).reshape(1, 2), i32(2, 3).reshape(1, 2)
    x16 = torch.zeros(2, k, dtype=torch.float16, device=DEV)
    cs, slots = torch.zeros(3, 32, 2, device=DEV), i32(0, 1, 2)
    freqs = torch.ones(32, dtype=torch.float64, device=DEV)
    table, ctx = i32(0, 1, 2, 3).reshape(1, 4), i32(5)
    long = i32(*([0] * 200)).reshape(1, 200)
    ws = q.attention_workspace(cache, rows, long)
    assert ws.numel() > 0
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    return [
        lambda: q.rope_angles(slots, freqs, out=cs), lambda: q.rope(rows, cs, out=out),
        lambda: q.kv_append(cache, kv, kv, slots, cs=cs), lambda: q.kv_read(cache, slots, k_out=kv, v_out=kv),
        lambda: q.kv_move(cache, src, dst),
        lambda: q.attention(cache, rows, table, ctx, out=out, workspace=none),
        lambda: q.attention(cache, rows, long, ctx, out=out, workspace=ws),
        lambda: q.attention(cache, many, table, ctx, out=more, workspace=none, max_ctx=64),
        lambda: q.dequant(w, G.Q4_K, n, k), lambda: q.dequant_f16(w, G.Q4_K, n, k),
        lambda: q.embed(w, G.Q4_K, n, k, slots), lambda: q.quantize(x, G.Q8_0),
        lambda: q.gemv(w, G.Q4_K, n, k, x1, out=y1), lambda: q.gemv(w, G.Q4_K, n, k, x, out=y),
        lambda: q.gemv(w8, G.Q8_0, n, k, x, out=y), lambda: q.gemv_multi([w, w], G.Q4_K, [n, n], k, [x, x]),
        lambda: q.gemv_multi([w8, w8], G.Q8_0, [n, n], k, [x1, x1]),
        lambda: q.gemv_pass([(w, G.Q4_K, n, k, x1[0], y1[0], 0), (w8, G.Q8_0, n, k, x1[0], y[0], 1)]),
        lambda: q.gemm_prefill(w, G.Q4_K, n, k, x16),
    ]


def test_errors_of_others_stay_theirs(hip):
    calls = every()
    for call in calls:
        call()
    torch.cuda.synchronize()
    for i, call in enumerate(calls):
        bad = hip.hipSetDevice(99)
        assert bad != 0
        call()
        assert hip.hipGetLastError() == bad, i
    torch.cuda.synchronize()
