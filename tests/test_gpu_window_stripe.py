"""Windows below the number of shards in the stripe layout, with shards whose last row is a query tile
of its own: a key can lie between the windows of a block's two query tiles. Definition, inputs and
tolerances are those of test_gpu_window.py, but for float32 gradients: a query that sees one key has
dP - delta = 0 in exact arithmetic, and its gradients are what two float32 sums of dh = 64 products
differ by. Each is off by at most dh * 2^-24 * sum |dO v| (64 * 2^-24 * 41 for normal numbers: 1.6e-4),
so an element by less than 2 * 1.6e-4 * scale (1/8) * |k| (2.5 in the mean square's worst case of a
row) = 1e-4: the absolute term that test_gpu_window.py has for bf16 on the same grounds, added to its
1e-5."""
import numpy as np
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
import test_gpu_window as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


# dtype, layout, D, lens, varlen, hq, hkv, dh, window, sinks
CASES = [
    (G.BF16, "stripe", 2, [258], False, 2, 1, 128, 1, 0),
    (G.BF16, "stripe", 3, [387], False, 2, 2, 128, 1, 0),
    (G.BF16, "stripe", 4, [516, 516], False, 4, 2, 64, 1, 0),
    (G.BF16, "stripe", 4, [516], False, 4, 2, 128, 2, 1),
    (G.BF16, "stripe", 4, [516], False, 4, 2, 128, 3, 0),
    (G.BF16, "stripe", 2, [770], False, 8, 2, 128, 1, 128),
    (G.BF16, "stripe", 8, [8 * 385], False, 2, 1, 64, 5, 3),
    (G.BF16, "stripe", 8, [8 * 129, 40, 0, 8 * 130, 8, 8 * 385], True, 2, 1, 128, 4, 2),
    (G.BF16, "stripe", 64, [64 * 129], False, 1, 1, 64, 40, 0),
    (G.F32, "stripe", 4, [516], False, 4, 2, 64, 2, 1),
    (G.BF16, "zigzag", 4, [4 * 386], False, 2, 1, 64, 2, 0),
    (G.BF16, "basic", 3, [387], False, 2, 1, 64, 1, 1),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0])[6:]}_{c[1]}_D{c[2]}_{max(c[3])}_dh{c[7]}_w{c[8]}_s{c[9]}")
def test_windows_below_the_number_of_shards(case, monkeypatch):
    if case[0] == G.F32:
        def check(got, ref, dt, what):
            off, size = np.linalg.norm(got - ref), np.linalg.norm(ref)
            assert off <= 1e-5 * size + 1e-4 * ref.size ** 0.5, f"{what}: off by {off:.3e} of {size:.3e}"
        monkeypatch.setattr(G, "check_l2", check)
    G.test_window_forward_and_backward(case)
