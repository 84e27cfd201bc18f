"""What the tolerance of FP8 sums on normal values tells apart, with mistakes planted in the
64-bit form: a step under another step's scales, a chunk of a row lost or read twice. No GPU."""
import numpy as np
import pytest

import llm_reference as ref


def _values(rows, K, seed, uneven):
    r = np.random.RandomState(seed)
    v = r.standard_normal((rows, K))
    v = ref.E4M3[ref.e4m3_codes(v * 100)] / 100
    s = np.exp2(r.randint(-6, 7, (rows, K // 128))) if uneven else np.ones((rows, K // 128))
    return v, s


def _outside(wrong_a, a, b):
    """Share of the outputs that a product with wrong_a puts out of the tolerance of a b^T."""
    c, s = ref.product(a, b)
    return (np.abs(wrong_a @ b.T - c) > ref.fp8_mfma_tolerance(a, b, c, s)).mean()


@pytest.mark.parametrize("K", [1152, 1408, 2048])
@pytest.mark.parametrize("first,last,back", [(8, None, 8), (8, 9, 4), (4, 8, 4), (1, 2, 1), (-1, None, 1)])
def test_scales_of_another_step(K, first, last, back):
    """Steps first .. last - 1 under the scales of `back` steps before."""
    v, s = _values(40, K, 1, True)
    b, _ = _values(50, K, 2, False)
    stale = s.copy()
    steps = np.arange(s.shape[1])[first:last]
    stale[:, steps] = s[:, steps - back]
    spread = lambda t: v * np.repeat(t, 128, 1)  # noqa: E731
    assert _outside(spread(stale), spread(s), b) > 0.4
    assert _outside(spread(s), spread(s), b) == 0


@pytest.mark.parametrize("K", [384, 1664, 4096])
def test_chunk_of_a_row(K):
    """16 codes lost, or those of the step before in their place."""
    a, _ = _values(40, K, 3, False)
    b, _ = _values(50, K, 4, False)
    for value in (0.0, a[:, 128:144]):
        wrong = a.copy()
        wrong[:, 256:272] = value
        assert _outside(wrong, a, b) > 0.8
