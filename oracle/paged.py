"""Oracle of the rotary and paged-cache calls: their definitions in 64 bits,
one sequence and one head at a time, on CPU tensors (torch, for bfloat16).

TEST INFRASTRUCTURE ONLY; shares no code with the product path.
"""
from __future__ import annotations

import math

import torch


def rope(x, positions, freqs, layout="half", attn_factor=1.0, inverse=False):
    """x [T, H, d] -> fp64 [T, H, d], pair by pair as a complex product."""
    y = x.double().clone()
    for i, f in enumerate(freqs.double().tolist()):
        a, b = ((i, i + freqs.numel()) if layout == "half"
                else (2 * i, 2 * i + 1))
        for t, p in enumerate(positions.tolist()):
            z = complex(math.cos(p * f), math.sin(p * f)) * attn_factor
            z = z.conjugate() if inverse else z
            xa, xb = x[t, :, a].double(), x[t, :, b].double()
            y[t, :, a] = xa * z.real - xb * z.imag
            y[t, :, b] = xa * z.imag + xb * z.real
    return y


def rope_bound(x, freqs, layout, attn_factor, angle):
    """Bound of the fp32 part of a rotation's error, per element: `angle` for
    the angle (radians), 2^-22 for cosine and sine (twice the library's 2
    ulp), 2^-23 for the two products and their sum, each relative to
    |x_a| + |x_b|."""
    e = (angle + 2.0 ** -22 + 2.0 ** -23) * attn_factor
    y = torch.zeros_like(x, dtype=torch.float64)
    n = freqs.numel()
    i = torch.arange(n)
    a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    s = x[..., a].double().abs() + x[..., b].double().abs()
    y[..., a] = s * e
    y[..., b] = s * e
    return y


def quantised(x):
    """Codes and scale of rows of the last axis, in the 32-bit arithmetic
    that defines them."""
    a = x.float().abs().amax(-1)
    scale = a * (torch.ones(()) / 127.0)
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    q = (x.float() / safe[..., None]).round().clamp(-127, 127).to(torch.int8)
    return q, scale


def places(cu, kv_lens, table, page):
    """(token, sequence, position, page id, slot) of every new token."""
    out = []
    for b, n in enumerate(kv_lens):
        m = cu[b + 1] - cu[b]
        for i in range(m):
            p = n - m + i
            out.append((cu[b] + i, b, p, int(table[b][p // page]), p % page))
    return out


def attn(q, k_pages, v_pages, table, cu, kv_lens, *, causal=True, scale=None,
         k_scale=None, v_scale=None):
    """Returns out fp64 [T, hq, d] (NaN in rows of no sequence), lse fp64
    [hq, T], and the bound of the device's error in out, per element."""
    t, hq, d = q.shape
    _, page, hkv, _ = k_pages.shape
    group = hq // hkv
    scale = d ** -0.5 if scale is None else scale
    out = torch.full((t, hq, d), math.nan, dtype=torch.float64)
    tol = torch.zeros((t, hq, d), dtype=torch.float64)
    lse = torch.full((hq, t), math.nan, dtype=torch.float64)
    int8 = k_scale is not None
    u_p = 2.0 ** -11 if int8 or q.dtype == torch.float16 else 2.0 ** -8
    u_o = 2.0 ** -11 if q.dtype == torch.float16 else 2.0 ** -8
    for b, n in enumerate(kv_lens):
        m = cu[b + 1] - cu[b]
        pos = torch.arange(n)
        ids = torch.as_tensor(table[b])[pos // page].long()
        k, v = k_pages[ids, pos % page].double(), v_pages[ids, pos % page].double()
        if int8:
            k = k * k_scale[ids, :, pos % page].double()[..., None]
            v = v * v_scale[ids, :, pos % page].double()[..., None]
        for i in range(m):
            seen = n - m + i + 1 if causal else n
            row = cu[b] + i
            for h in range(hq):
                if seen <= 0:
                    out[row, h] = 0
                    lse[h, row] = -math.inf
                    continue
                kk, vv = k[:seen, h // group], v[:seen, h // group]
                qq = q[row, h].double()
                s = kk @ qq * scale
                z = torch.logsumexp(s, 0)
                p = torch.exp(s - z)
                out[row, h] = p @ vv
                lse[h, row] = z
                # each score: fp32 sums of d products and a few roundings;
                # each weight: its rounding to 16 bits (u_p), 2^-21 for the
                # exponential, and 2^-25 of the largest for subnormals
                # (INT8: of twice the largest V scale times 127)
                ds = float((kk.abs() @ qq.abs()).max()) * scale * (d + 8) * 2.0 ** -24
                w = (u_p + 2.0 ** -20 + 2 * ds) * (p @ vv.abs())
                top = p.max()
                big = vv.abs().amax() if int8 else vv.abs().amax(0)
                w = w + 2.0 ** -25 * seen * top * (2.0 * big if int8 else big)
                # fp32 sums over the keys
                w = w + seen * 2.0 ** -24 * (p @ vv.abs())
                tol[row, h] = w + u_o * out[row, h].abs() + 2.0 ** -25
    return out, lse, tol
