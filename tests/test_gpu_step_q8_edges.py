"""Products of Q8_0 activations where a matrix ends inside a 16-byte chunk: poison
follows the weights and the activations directly (0xff: a scale that is not a number).
|y - exact| <= 2e-5 sum |w x|."""
import numpy as np
import pytest

import oracle
import qmm_inputs as G

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_matmul_amd as q  # noqa: E402

DEV = "cuda:0"
TOL = 2e-5


def between_poison(a, before=64):
    """The bytes of a on the device, 16-byte aligned, 0xff on both sides."""
    buf = torch.full((before + a.size + 4096,), 255, dtype=torch.uint8, device=DEV)
    view = buf[before:before + a.size]
    view.copy_(torch.from_numpy(np.ascontiguousarray(a).reshape(-1)))
    assert view.data_ptr() % 16 == 0
    return view


# short rows, several to an item; one segment; several; more than eight, the last round
# with waves behind the row's end (units of 32 elements, 64 to a segment; Q6_K of 64)
@pytest.mark.parametrize("t,blocks", [
    (t, b) for t in (G.Q8_0, G.Q4_0, G.Q5_0) for b in (1, 5, 17, 31, 33, 63, 65, 127, 449, 513, 579, 700, 1100)]
    + [(G.Q6_K, b) for b in (1, 3, 5, 9, 15, 17, 33, 113, 129, 145, 261)])
def test_matrices_that_end_inside_a_chunk(t, blocks):
    k = blocks * G.BLOCK_ELEMS[t]
    rng = np.random.default_rng(100 * t + blocks)
    for n in (1, 3, 7):                        # rows of 2 mod 4 bytes: no multiple of 16
        w = G.gen_weights(t, n, k, seed=n + blocks)
        wd = between_poison(w)
        assert w.size % 16 or blocks % 8 == 0
        W = oracle.dequant(t, w, n, k).astype(np.float64)
        for batch in (1, 2, 5):
            x = oracle.quantize(G.Q8_0, rng.standard_normal((batch, k)).astype(np.float32))
            X = oracle.dequant(G.Q8_0, x, batch, k).astype(np.float64)
            xd = between_poison(x).view(batch, -1)
            y = q.gemv_q8(wd, t, n, k, xd).cpu().numpy()
            assert np.all(np.abs(y - X @ W.T) <= TOL * (np.abs(X) @ np.abs(W).T))
