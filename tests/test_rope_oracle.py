"""The rotating operators' reference against closed forms, and torch's e4m3 rounding."""
import numpy as np
import pytest
import torch

from tests import rope_oracle as ro


@pytest.mark.parametrize("interleaved", [False, True])
def test_scores_of_rotated_vectors_depend_on_distances(interleaved):
    """In 64 bits, q turned by p against k turned by t is q turned by p - t against k."""
    rng = np.random.default_rng(1)
    tab = ro.table(200, 32).astype(np.float64)
    q, k = rng.standard_normal((2, 1, 64))

    def at(x, p):
        return ro.rotate(x, tab, [p], 64, 16, interleaved)

    # the table's entries are off by 2^-25 each
    assert abs((at(q, 150) @ at(k, 60).T - at(q, 90) @ k.T).item()) < 64 * 2.0 ** -22
    back = ro.rotate(at(q, 150), tab, [150], 64, 16, interleaved, inverse=True)
    assert np.abs(back - q).max() < 2.0 ** -21


def test_pair_by_hand():
    tab = np.array([[1, 1] + [1] * 6 + [0] * 8, [0, 1] + [1] * 6 + [1, 0] + [0] * 6], np.float32)
    x = np.arange(64, dtype=np.float64)[None]
    y = ro.rotate(x, tab, [1], 64, 8, True)
    assert (y[0, 8], y[0, 9]) == (-9, 8) and np.array_equal(np.delete(y, [8, 9]), np.delete(x, [8, 9]))
    y = ro.rotate(x, tab, [1], 64, 8, False)
    assert (y[0, 8], y[0, 16]) == (-16, 8) and np.array_equal(np.delete(y, [8, 16]), np.delete(x, [8, 16]))
    assert np.array_equal(ro.rotate(x, tab, [-1], 64, 8, False), x)


def test_codes_are_torchs():
    v = np.concatenate([np.linspace(-448, 448, 20001), np.linspace(-0.1, 0.1, 20001)]).astype(np.float32)
    mids = (ro.FINITE[1:] + ro.FINITE[:-1]) / 2
    v = np.concatenate([v, mids.astype(np.float32)])
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    got = ro.nearest_codes(v)
    assert np.array_equal(got, want) and np.array_equal(np.signbit(got), np.signbit(want))
