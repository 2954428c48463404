"""How exact the positions' sines and cosines are, seen by themselves."""
import numpy as np
import pytest
import torch

from test_gpu_serving import dev, ra  # noqa: F401  (ra: the module's fixture)

pytestmark = pytest.mark.gpu


def sines(ra, pos, freq, fn):  # noqa: F811
    """(cos, sin) as the kernels have them: pairs (1, 0), whose products with them are exact."""
    x = torch.zeros((len(pos), 1, 2 * len(freq)), device="cuda")
    x[..., :len(freq)] = 1
    y = fn(x, None, dev(pos), freq)[0][:, 0].double().cpu().numpy()
    return y[:, :len(freq)], y[:, len(freq):]


def close(got, want, angle):
    """One unit in the last place of the sine or cosine, the argument's rounding (half of 2^-26 half turns, and what is
    cut off below 2^-33), what the table cuts off (2^-64 turns, times a position of at most 2^31), and the rounding of
    position times frequency in 64 bits here and in the table."""
    bound = np.spacing(np.abs(want).astype(np.float32)) + np.pi * (2.0 ** -27 + 2.0 ** -33 + 2.0 ** -32) + \
        np.abs(angle) * 2.0 ** -51
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())


@pytest.mark.parametrize("T", [2000, 5000])  # a warp a token, and the ring
def test_angles_keep_the_bits_of_a_float(ra, T):  # noqa: F811
    rng = np.random.default_rng(T)
    pos, freq = rng.integers(0, 1 << 17, T), 10000.0 ** (-np.arange(32) / 32)
    angle = pos[:, None] * freq
    for fn, sign in ((ra.rope_fwd, 1), (ra.rope_bwd, -1)):
        c, s = sines(ra, pos, freq, fn)
        close(c, np.cos(angle), angle)
        close(s, sign * np.sin(angle), angle)


def test_angles_of_negative_frequencies(ra):  # noqa: F811
    """A frequency below zero turns the other way, as exactly, slow ones at far positions too."""
    pos = np.array([2**31 - 1, 2**31 - 12345, -2**31, 10**9 + 7, 12345, 1], np.int64)
    freq = -np.array([1e-9, 3.7e-10, 2e-6, 0.5, 1.0, 7.25, 1e-12, 0.0])
    angle = pos[:, None] * freq
    for fn, sign in ((ra.rope_fwd, 1), (ra.rope_bwd, -1)):
        c, s = sines(ra, pos, freq, fn)
        close(c, np.cos(angle), angle)
        close(s, sign * np.sin(angle), angle)
