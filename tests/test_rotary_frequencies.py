"""The range of rotary frequencies: the angle's bound holds for every frequency that is accepted."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

FAKE = 0x10000
# 1 / (2 pi) to 80 digits: times 2^32 radians and a position of 2^31 still good to 1e-60 turns
PER_RADIAN = Fraction(
    "0.15915494309189533576888376337251436203445964574045644874766734405889679763422653")


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_53_gb300 import build
    path = build.build()
    import paged_kv_cache_53_gb300 as pa
    pa.lib(path)
    return pa


@pytest.mark.parametrize("freq", [2.0 ** 32 * (1 + 2.0 ** -52), -2.0 ** 33, 1e300, -1.7e308])
def test_frequencies_past_the_range_are_refused(pa, freq):
    lib = pa.lib()
    inv = (ctypes.c_double * 2)(1.0, freq)
    axis = (ctypes.c_int32 * 2)(0, 0)
    rc = lib.pa_rotary_append(FAKE, FAKE * 2, 256, FAKE, 64, FAKE, 64, FAKE, FAKE, None, FAKE, 4,
                              FAKE, FAKE, FAKE, 1, inv, axis, 4, 0, 1, 1, 4, 1, 64, 16, 8, 0, None)
    msg = lib.pa_last_error_string().decode()
    assert rc == 1 and "pa_rotary_append" in msg and "inv_freq[1]" in msg


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_up_to_the_range(pa, interleaved):
    """fp32, against exact turn counts.  The angle: 2^-26 + 2^-31 turns; sine and cosine add 2^-24
    each, each product and the sum round by 2^-24."""
    pa.get_status()
    freqs = [2.0 ** 32, -(2.0 ** 32), 2.0 ** 32 - 0.7, 4.1e9, 123456789.125, 2.0 ** 31 / 3, 1e6 / 7,
             6.283185307179586, 1.0, 1e-4, 1e-12, 5e-324]
    pos = [0, 1, -1, 7, 99991, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, -(2 ** 31)]
    half, t, d = len(freqs), len(pos), 64
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(t, h, d, generator=g, device="cuda") for h in (2, 1, 1))
    kc, vc = (torch.zeros(2, 1, 16, d, device="cuda") for _ in range(2))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.empty_like(q)
    pa.rotary_append(out, q, k, v, kc, vc, i32([[0, 1]]), i32([0, t]), i32([t]), i32([pos]),
                     pa.Rotary(freqs, interleaved=interleaved))
    torch.cuda.synchronize()
    assert pa.get_status() == 0
    turns = np.array([[float(Fraction(f) * p * PER_RADIAN % 1) for f in freqs] for p in pos])
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    bound = 2 * np.pi * (2.0 ** -26 + 2.0 ** -31) + 3 * 2.0 ** -24
    for x, got in ((q, out), (k, kc[0, :, :t].transpose(0, 1))):
        x, got = x.double().cpu().numpy(), got.double().cpu().numpy()
        tol = bound * (np.abs(x[..., a]) + np.abs(x[..., b]))
        assert (np.abs(got[..., a] - (x[..., a] * c - x[..., b] * s)) <= tol).all()
        assert (np.abs(got[..., b] - (x[..., b] * c + x[..., a] * s)) <= tol).all()
