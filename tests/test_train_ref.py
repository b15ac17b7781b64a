"""The 64-bit forms that the GPU tests compare with: gradients against differences, random bits against a direct
evaluation (CPU)."""
import numpy as np
import pytest

from tests import train_ref as ref


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_gradient_is_the_difference(kind):
    rng = np.random.RandomState(1)
    g, v, dh = (rng.randn(2000) * s for s in (3, 2, 1))
    got = ref.gated_grad(dh, g, v, kind)
    e = 1e-6  # central differences: third derivatives times e^2 / 6, and 2^-53 / e from rounding
    for name, d in (("dg", (ref.gated(g + e, v, kind)[0] - ref.gated(g - e, v, kind)[0]) / (2 * e)),
                    ("dv", (ref.gated(g, v + e, kind)[0] - ref.gated(g, v - e, kind)[0]) / (2 * e))):
        assert np.max(np.abs(got[name][0] - dh * d)) < 1e-7
    assert np.all(got["h"][0] == ref.gated(g, v, kind)[0])


def test_activations_are_what_they_are_called():
    import torch
    x = torch.linspace(-20, 20, 4001, dtype=torch.float64)
    one = np.ones(4001)
    for kind, f in (("silu", torch.nn.functional.silu), ("gelu", lambda t: torch.nn.functional.gelu(t, approximate="tanh"))):
        assert np.max(np.abs(ref.gated(x.numpy(), one, kind)[0] - f(x).numpy())) < 1e-13


def test_random_bits():
    m = 2 ** 32

    def one(key, i):
        h = ((i * 0x9E3779B1 % m) ^ (i >> 32)) + key
        h %= m
        h = (h ^ (h >> 16)) * 0x85EBCA6B % m
        h = (h ^ (h >> 13)) * 0xC2B2AE35 % m
        return h ^ (h >> 16)

    at = [0, 1, 2, 12345, 2 ** 31 + 7, 2 ** 32 - 1, 2 ** 32, 2 ** 33 + 5]
    for key in (0, 1, 0xFFFFFFFF, 987654321):
        assert ref.random_bits(key, at).tolist() == [one(key, i) for i in at]
    r = ref.random_bits(3, np.arange(1 << 16))
    assert len(np.unique(r)) == 1 << 16  # for one key the bits are a permutation of the places
    for half in (r & 0xFFFF, r >> 16):   # mean of 2^16 uniform values: 6 standard deviations of 2^16 / sqrt(12 * 2^16)
        assert abs(half.mean() - 32767.5) < 6 * 65536 / np.sqrt(12 * 65536)


def test_codes():
    import torch
    q = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(q).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.decode(q), t, equal_nan=True)
