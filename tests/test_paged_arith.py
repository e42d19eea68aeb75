"""Arithmetic of the paged-cache kernels, modelled on the host in IEEE
float32: the exponential on the FMA pipe and the INT8 scale."""
import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "prefill_blockwise_int8_b200", "csrc")
F = np.float32


def _fma(a, b, c):
    # the product of two floats is exact in float64, and the sum is off by
    # 2^-53 of it before it rounds to float32
    return (a.astype(np.float64) * np.asarray(b, np.float64) +
            np.asarray(c, np.float64)).astype(F)


def _ex2_poly(x):
    """ex2_poly2 of attn_common.cuh with the coefficients of its source."""
    src = open(os.path.join(CSRC, "attn_common.cuh")).read()
    body = src[src.index("float2 ex2_poly2"):]
    body = body[:body.index("\n}")]
    found = re.findall(r"make_float2\((0x1\.[0-9a-f]+p-\d+)f, \1f\)", body)
    coef = [F(float.fromhex(c)) for c in found]
    assert len(coef) >= 4 and "make_float2(1.0f, 1.0f)" in body
    x = np.maximum(x.astype(F), F(-127))
    magic = F(12582912.0)  # 1.5 * 2^23
    t = x + magic
    n = t - magic
    f = _fma(n, F(-1), x)
    p = np.full_like(f, coef[0])
    for c in coef[1:] + [F(1)]:
        p = _fma(f, p, c)
    return ((t.view(np.int32) << 23) + p.view(np.int32)).view(F)


def test_exponential_on_the_fma_pipe():
    # as good as the exponential unit's 2^-22 within half of it: the bound of
    # the attention's outputs grants 2^-21
    x = np.linspace(-125.9, 24.0, 3_000_001).astype(F)
    err = np.abs(_ex2_poly(x).astype(np.float64) /
                 np.exp2(x.astype(np.float64)) - 1)
    assert err.max() <= 2.0 ** -21
    # far below: nothing, never negative or large
    low = np.linspace(-300.0, -126.0, 100_001).astype(F)
    assert (_ex2_poly(low) >= 0).all() and (_ex2_poly(low) <= 2.0 ** -125).all()
    assert (_ex2_poly(np.array([-127.0, -np.inf, -1e30], F)) == 0).all()
    assert (_ex2_poly(np.arange(-126, 25).astype(F)) ==
            np.exp2(np.arange(-126, 25)).astype(F)).all()


def _halves(dtype):
    """Every positive finite value of fp16 or bf16, as float32."""
    bits = np.arange(1, 1 << 15, dtype=np.uint32)
    if dtype == "fp16":
        x = bits.astype(np.uint16).view(np.float16).astype(F)
    else:
        x = (bits << 16).view(F)
    return x[np.isfinite(x)]


def test_int8_scale_against_the_quantisers():
    # the append's scale a * fl(1 / 127) and the block quantiser's fl(a / 127):
    # at most one step apart for every row maximum there is, and the row
    # maximum's code is 127 under both
    inv = F(1) / F(127)
    for dtype in ("fp16", "bf16"):
        a = _halves(dtype)
        mul, div = a * inv, a / F(127)
        assert (np.abs(mul - div) <= np.spacing(div)).all()
        assert (mul > 0).all()
        for s in (mul, div):
            assert (np.rint(a / s) == 127).all()
    # so a code moves by one at most, and only where x / scale lies within
    # 127 * 2^-22 of a half
    rng = np.random.default_rng(0)
    xs = _halves("fp16")
    for a in rng.choice(xs[xs > 2.0 ** -14], 200):
        x = xs[xs <= a]
        q = x / (a * inv)
        c, d = np.rint(q), np.rint(x / (a / F(127)))
        moved = c != d
        assert (np.abs(c - d) <= 1).all()
        assert (np.abs(np.abs(q[moved] - np.floor(q[moved])) - 0.5) <=
                127 * 2.0 ** -22).all()
