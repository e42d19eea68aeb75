"""Cases of the serving operators around the paged KV cache: rotary positions
(`tilemix_rope`), appending new tokens to the pages (`tilemix_paged_append`)
and attention of new tokens over the pages (`tilemix_attn_paged`).

`run` computes an operator in its plain form (elementary torch operations in
32 bits, angles in 64), or, where `own` is true, calls the framework.

Layouts: tensors of tokens are [T, heads, head_dim] over the concatenated
batch (`cu_seqlens`); pages are [num_pages, page_size, kv_heads, head_dim]
and a sequence's position p lies in page `page_table[b][p // page_size]`, slot
`p % page_size`; scales of INT8 pages are [num_pages, kv_heads, page_size].
"""
import math
import random

import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _rope(name, tokens, hq, hkv, d, rot, **kw):
    return dict(dict(name=name, op="rope", tokens=tokens, hq=hq, hkv=hkv, d=d,
                     rot=rot, dtype="bf16", layout="half", inverse=False,
                     fused_qkv=True, attn_factor=1.0, max_pos=131072), **kw)


def _append(name, batch, new_min, new_max, ctx_min, ctx_max, hq, hkv, d, **kw):
    return dict(dict(name=name, op="append", batch=batch, new_min=new_min,
                     new_max=new_max, ctx_min=ctx_min, ctx_max=ctx_max, hq=hq,
                     hkv=hkv, d=d, rot=0, page=16, kv="same", dtype="bf16",
                     layout="half", lens=1), **kw)


def _attn(name, batch, new_min, new_max, ctx_min, ctx_max, hq, hkv, d, **kw):
    return dict(dict(name=name, op="attn", batch=batch, new_min=new_min,
                     new_max=new_max, ctx_min=ctx_min, ctx_max=ctx_max, hq=hq,
                     hkv=hkv, d=d, page=16, kv="same", dtype="bf16",
                     causal=True, lens=1), **kw)


def listed():
    return [
        # one decode step of 16 sequences: Q and K are slices of the fused
        # projection's output; a small call, where latency counts
        _rope("rope_step_16", 16, 32, 8, 128, 128),
        # the bench workload's prefill (8 x 4096 tokens, 24 / 8 heads)
        _rope("rope_prefill_32768", 32768, 24, 8, 128, 128, dtype="fp16"),
        # decode step: rotation of q and k and the write into 16-bit pages
        _append("append_step_64", 64, 1, 1, 1, 8191, 32, 8, 128, rot=128),
        # a prefilled batch (16 sequences, 512..8192) into 16-bit pages, with
        # half of each head rotated, interleaved pairs
        _append("append_varlen_rope", 16, 512, 8192, 0, 0, 28, 4, 128,
                rot=64, layout="interleaved", page=32, dtype="fp16", lens=2),
        # the INT8 cache of 2 x 16384 tokens with 32 KV heads, written once
        _append("append_int8_prefill", 2, 16384, 16384, 0, 0, 32, 32, 128,
                kv="int8", page=128, dtype="fp16"),
        # one token of one sequence over a short cache: the smallest call
        _attn("step_b1", 1, 1, 1, 4095, 4095, 32, 8, 128),
        # one token of 64 sequences of very different lengths
        _attn("step_b64_ragged", 64, 1, 1, 1023, 32767, 32, 8, 128, lens=3),
        # one token over the INT8 cache, one query head per KV head
        _attn("step_int8", 8, 1, 1, 8191, 16383, 32, 32, 128, kv="int8",
              page=128, dtype="fp16", lens=4),
        # a few drafted tokens verified at once, 7 query heads a KV head,
        # odd lengths
        _attn("verify_5_h28x4", 16, 5, 5, 507, 8187, 28, 4, 128, page=64,
              dtype="fp16", lens=2),
        # a prompt's chunk over a long cache: the largest call
        _attn("chunk_2048_of_32768", 1, 2048, 2048, 30720, 30720, 32, 8, 128,
              page=128),
        # chunks of several prompts over an INT8 cache, 24 / 8 heads
        _attn("chunk_int8_ragged", 8, 1, 1024, 512, 8192, 24, 8, 128,
              kv="int8", page=64, dtype="fp16", lens=6),
        # a decoder's tokens over an encoder's 1500 states (no causal mask)
        _attn("cross_448_1500", 8, 448, 448, 1500, 1500, 16, 16, 64,
              page=32, dtype="fp16", causal=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo),
                                                          math.log(hi)))))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(("rope", "append", "append", "attn", "attn", "attn"))
    dtype = rng.choice(("fp16", "bf16"))
    d = rng.choice((64, 128, 128))
    hkv = rng.choice((1, 2, 4, 8))
    hq = hkv * rng.choice((1, 2, 3, 4, 5, 7, 8))
    if op == "rope":
        layout = rng.choice(("half", "interleaved"))
        d = rng.choice((64, 80, 96, 128, 256))
        return _rope("", _log_int(rng, 1, 32768 * 16 // max(16, hq)), hq, hkv,
                     d, rng.choice([r for r in (16, 32, 64, 96, 128, 256)
                                    if r <= d]),
                     dtype=dtype, layout=layout, inverse=rng.random() < 0.3,
                     fused_qkv=rng.random() < 0.5,
                     attn_factor=rng.choice((1.0, 1.2079441541679836)),
                     max_pos=rng.choice((4096, 131072, 1048576)))
    batch = _log_int(rng, 1, 48)
    page = rng.choice((16, 32, 64, 128))
    kv = rng.choice(("same", "int8"))
    lens = rng.randrange(1 << 20)
    if op == "append":
        new = _log_int(rng, 1, 32768 // batch)
        return _append("", batch, rng.randint(0, new), new, 0, 3000, hq, hkv, d,
                       rot=0 if kv == "int8" else rng.choice((0, 32, d)),
                       page=page, kv=kv, dtype=dtype, lens=lens,
                       layout=rng.choice(("half", "interleaved")))
    if rng.random() < 0.4:  # single tokens
        new_lo = new_hi = 1
    else:
        new_hi = _log_int(rng, 2, 1200)
        new_lo = rng.randint(0, new_hi)
    # keys a sequence, so that the whole stays below the largest listed case
    most = int(max(1, min(16384, 1.5e6 / batch / max(1, hkv // 4),
                          1.2e9 / (batch * new_hi * hq))))
    ctx = _log_int(rng, 1 if rng.random() < 0.1 else min(64, most), most)
    return _attn("", batch, new_lo, new_hi, rng.randint(0, ctx), ctx, hq, hkv,
                 d, page=page, kv=kv, dtype=dtype, lens=lens,
                 causal=rng.random() < 0.8)


def _lens(case):
    """(new tokens, cached tokens before them) of each sequence.  Without a
    causal mask the cache is an encoder's: the new tokens are not in it.  The
    first sequence has the most of both."""
    r = random.Random(case["lens"])
    rest = range(case["batch"] - 1)
    new = [r.randint(case["new_min"], case["new_max"]) for _ in rest]
    ctx = [r.randint(case["ctx_min"], case["ctx_max"]) for _ in rest]
    return [case["new_max"]] + new, [case["ctx_max"]] + ctx


def _kv_lens(case):
    new, ctx = _lens(case)
    if case["op"] == "attn" and not case["causal"]:
        return ctx
    return [n + c for n, c in zip(new, ctx)]


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        n = case["tokens"]
        return {"bytes": 4.0 * n * (hq + hkv) * d + 4 * n,
                "flops": 3.0 * n * (hq + hkv) * case["rot"]}
    new, _ = _lens(case)
    lens = _kv_lens(case)
    n = sum(new)
    tables = 4 * sum(-(-x // case["page"]) for x in lens)
    if case["op"] == "append":
        rows = 2 * n * hkv
        out = rows * (d + 4 if case["kv"] == "int8" else 2 * d)
        q = 4 * n * hq * d if case["rot"] else 0
        return {"bytes": float(2 * rows * d + out + q + 4 * n),
                "flops": 3.0 * n * (hkv + hq) * case["rot"] + 2.0 * rows * d}
    e = d + 4 if case["kv"] == "int8" else 2 * d
    if case["causal"]:
        pairs = sum(m * (x - m) + m * (m + 1) // 2 for m, x in zip(new, lens))
    else:
        pairs = sum(m * x for m, x in zip(new, lens))
    live = sum(x for m, x in zip(new, lens) if m)
    return {"bytes": float(2 * live * hkv * e + n * hq * (4 * d + 4) + tables),
            "flops": 4.0 * d * hq * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(gen, shape, dtype, outliers=False):
    """N(0, 1) with, where asked, 4 of each head's channels scaled by 20 (the
    outlier channels that keys and queries of trained models have)."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if outliers:
        at = torch.rand(shape[-2:], generator=gen, device="cuda")
        top = at.topk(4, dim=-1).indices
        x.mul_(torch.ones(shape[-2:], device="cuda").scatter_(-1, top, 20.0))
    return x.to(dtype)


def _frequencies(rot):
    """Radians per position: base 500000 with the wavelength-dependent
    scaling of long-context models (factor 8 beyond 8192 positions, blended
    between wavelengths of 2048 and 8192)."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 500000.0 ** (-2.0 * i / rot)
    wave = 2 * math.pi / f
    blend = ((8192.0 / wave - 1.0) / 3.0).clamp(0.0, 1.0)
    return ((1 - blend) * f / 8.0 + blend * f).cuda()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = _TYPES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s = {"case": case}
    if case["op"] == "rope":
        n = case["tokens"]
        if case["fused_qkv"]:
            # slices of the projection's output, tokens (hq + 2 hkv) d apart
            qkv = _normal(gen, (n, hq + 2 * hkv, d), t)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        else:
            s["q"] = _normal(gen, (n, hq, d), t)
            s["k"] = _normal(gen, (n, hkv, d), t)
        s["positions"] = torch.randint(0, case["max_pos"], (n,), generator=gen,
                                       device="cuda", dtype=torch.int32)
        s["freqs"] = _frequencies(case["rot"])
        return s
    new, _ = _lens(case)
    lens = _kv_lens(case)
    page = case["page"]
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    n = cu[-1]
    pages = [-(-x // page) for x in lens]
    total = sum(pages) + 3
    # the cache's pages in no order, unused table entries negative
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(new), max(1, max(pages))), -1, dtype=torch.int32,
                       device="cuda")
    at = 0
    for b, c in enumerate(pages):
        table[b, :c] = order[at:at + c]
        at += c
    s["page_table"], s["cu_seqlens"] = table, _ints(cu)
    s["kv_lens"] = _ints(lens)
    s["max_q_len"], s["max_kv_len"] = max(new), max(lens)
    if case["op"] == "append":
        shape = (total, page, hkv, d)
        scales = (total, hkv, page)
        if case["kv"] == "int8":
            for name in ("k", "v"):
                s[name + "_pages"] = torch.zeros(shape, dtype=torch.int8,
                                                 device="cuda")
                s[name + "_scale"] = torch.zeros(scales, device="cuda")
        else:
            for name in ("k", "v"):
                s[name + "_pages"] = torch.zeros(shape, dtype=t, device="cuda")
        qkv = _normal(gen, (n, hq + 2 * hkv, d), t)
        s["q"] = qkv[:, :hq]
        s["k"], s["v"] = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["freqs"] = _frequencies(case["rot"]) if case["rot"] else None
        return s
    s["q"] = _normal(gen, (n, hq, d), t, outliers=True)
    k = _normal(gen, (total, page, hkv, d), t, outliers=True)
    v = _normal(gen, (total, page, hkv, d), t)
    if case["kv"] == "int8":
        for name, x in (("k", k), ("v", v)):
            x8, scale = _quantised(x)
            s[name + "_pages"] = x8
            s[name + "_scale"] = scale.transpose(1, 2).contiguous()
    else:
        s["k_pages"], s["v_pages"] = k, v
    return s


def _quantised(x):
    """Codes and scales of rows of the last axis (symmetric, absmax / 127)."""
    x = x.float()
    scale = x.abs().amax(-1) / 127.0
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    codes = torch.round(x / safe[..., None]).clamp(-127, 127).to(torch.int8)
    return codes, scale


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rotated(x, positions, freqs, layout, factor=1.0, inverse=False):
    """x [T, H, d] with the first 2 * len(freqs) channels rotated, in 32 bits
    (angles and their cosines in 64)."""
    half = freqs.numel()
    angle = positions.double()[:, None] * freqs[None, :]
    c = (torch.cos(angle) * factor).float()[:, None, :]
    s = (torch.sin(angle) * factor).float()[:, None, :]
    if inverse:
        s = -s
    y = x.float()
    r = y[..., :2 * half]
    if layout == "half":
        a, b = r[..., :half], r[..., half:]
        r = torch.cat((a * c - b * s, b * c + a * s), -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    return torch.cat((r, y[..., 2 * half:]), -1).to(x.dtype)


def _places(s, n):
    """Sequence, position in the cache, page and slot of each new token."""
    case = s["case"]
    cu, lens = s["cu_seqlens"].long(), s["kv_lens"].long()
    t = torch.arange(n, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = lens[b] - (cu[b + 1] - cu[b]) + (t - cu[b])
    page = s["page_table"][b, pos // case["page"]].long()
    return b, pos, page, pos % case["page"]


def _plain_append(s):
    case = s["case"]
    k, v, q = s["k"], s["v"], None
    _, pos, page, slot = _places(s, k.shape[0])
    if case["rot"]:
        k = _rotated(k, pos, s["freqs"], case["layout"])
        q = _rotated(s["q"], pos, s["freqs"], case["layout"])
    for name, x in (("k", k), ("v", v)):
        if case["kv"] == "int8":
            codes, scale = _quantised(x)
            s[name + "_pages"][page, slot] = codes
            s[name + "_scale"][page, :, slot] = scale
        else:
            s[name + "_pages"][page, slot] = x
    return q


def _in_order(s, name, most):
    """The first `most` positions of every sequence, [B, most, hkv, d], in 32
    bits; positions past a sequence's end hold another's values."""
    p = s["case"]["page"]
    at = torch.arange(most, device="cuda")
    page = s["page_table"].clamp(min=0).long()[:, at // p]
    slot = (at % p)[None, :].expand_as(page)
    x = s[name + "_pages"][page, slot].float()
    if s["case"]["kv"] == "int8":
        x = x * s[name + "_scale"][page, :, slot][..., None]
    return x


def _plain_attn(s):
    case, q = s["case"], s["q"]
    n, hq, d = q.shape
    hkv, width, most = case["hkv"], s["max_q_len"], s["max_kv_len"]
    cu, lens = s["cu_seqlens"].long(), s["kv_lens"].long()
    if n == 0 or most == 0:
        return torch.zeros_like(q), torch.full((hq, n), -math.inf,
                                               device="cuda")
    new = cu[1:] - cu[:-1]
    i = torch.arange(width, device="cuda")
    rows = (cu[:-1, None] + i).clamp(max=n - 1)
    qp = q[rows].float().reshape(-1, width, hkv, hq // hkv, d)
    qp = qp.permute(0, 2, 3, 1, 4).flatten(2, 3)              # B hkv rN d
    k = _in_order(s, "k", most).permute(0, 2, 3, 1)           # B hkv d L
    x = torch.matmul(qp, k).mul_(d ** -0.5)                   # B hkv rN L
    last = lens[:, None].expand(-1, width) - 1                # last key seen
    if case["causal"]:
        last = last - new[:, None] + 1 + i
    last = last.repeat(1, hq // hkv)[:, None, :, None]
    x.masked_fill_(torch.arange(most, device="cuda") > last, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    w = x.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    v = _in_order(s, "v", most).permute(0, 2, 1, 3)           # B hkv L d
    o = torch.matmul(w, v) / torch.where(total > 0, total,
                                         torch.ones_like(total))
    lse = (top + total.log()).reshape(-1, hq, width)
    o = o.reshape(-1, hq, width, d)
    t = torch.arange(n, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    at = t - cu[b]
    return o[b, :, at].to(q.dtype), lse[b, :, at].t().contiguous()


def _plain(s):
    case = s["case"]
    if case["op"] == "rope":
        return [_rotated(s[x], s["positions"], s["freqs"], case["layout"],
                         case["attn_factor"], case["inverse"])
                for x in ("q", "k")]
    if case["op"] == "append":
        q = _plain_append(s)
        return [q] + [s[x] for x in ("k_pages", "v_pages", "k_scale",
                                     "v_scale") if x in s]
    return list(_plain_attn(s))


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own(s):
    import prefill_blockwise_int8_b200 as tm
    case = s["case"]
    layout = tm.ROPE_LAYOUTS[case.get("layout", "half")]
    if case["op"] == "rope":
        return list(tm.tilemix_rope(
            s["q"], s["k"], s["positions"], s["freqs"], layout=layout,
            attn_factor=case["attn_factor"], inverse=case["inverse"]))
    if case["op"] == "append":
        q = tm.tilemix_paged_append(
            s["k"], s["v"], s["page_table"], s["cu_seqlens"], s["kv_lens"],
            s["k_pages"], s["v_pages"], k_scale=s.get("k_scale"),
            v_scale=s.get("v_scale"), q=s["q"] if case["rot"] else None,
            freqs=s["freqs"], layout=layout)
        return [q] + [s[x] for x in ("k_pages", "v_pages", "k_scale",
                                     "v_scale") if x in s]
    lse = torch.empty((case["hq"], s["q"].shape[0]), device="cuda")
    out = tm.tilemix_attn_paged(
        s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["cu_seqlens"],
        s["kv_lens"], s["max_q_len"], s["max_kv_len"],
        k_scale=s.get("k_scale"), v_scale=s.get("v_scale"),
        causal=case["causal"], lse=lse)
    return [out, lse]


def run(state):
    """One call.  rope: [q, k] rotated; append: [rotated q or None, the pages,
    their scales] (INT8 codes are defined bit for bit, so they come back as
    they are stored, with the scales); attention: [out, lse]."""
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one sequence at a time
# ---------------------------------------------------------------------------

def _turn64(x, positions, freqs, layout, factor, sign):
    y = x.double().clone()
    n = freqs.numel()
    z = torch.polar(torch.full((), factor, dtype=torch.float64, device="cuda")
                    .expand(positions.numel(), n).contiguous(),
                    sign * positions.double()[:, None] * freqs)[:, None]
    i = torch.arange(n, device="cuda")
    re, im = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    w = torch.complex(y[..., re], y[..., im]) * z
    y[..., re], y[..., im] = w.real, w.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return [_turn64(s[x], s["positions"], s["freqs"], case["layout"],
                        case["attn_factor"], -1.0 if case["inverse"] else 1.0)
                for x in ("q", "k")]
    cu, lens = s["cu_seqlens"].tolist(), s["kv_lens"].tolist()
    p = case["page"]
    table = s["page_table"].tolist()
    if case["op"] == "append":
        q = s["q"].double().clone() if case["rot"] else None
        int8 = case["kv"] == "int8"
        pools = {x: s[x + "_pages"].double() for x in "kv"}
        scales = {x: s[x + "_scale"].double() for x in "kv"} if int8 else {}
        for b, x in enumerate(lens):
            rows = slice(cu[b], cu[b + 1])
            m = cu[b + 1] - cu[b]
            if m == 0:
                continue
            pos = torch.arange(x - m, x, device="cuda")
            page = s["page_table"][b].long()[pos // p]
            for name in "kv":
                y = s[name][rows].double()
                if case["rot"] and name == "k":
                    y = _turn64(s["k"][rows], pos, s["freqs"], case["layout"],
                                1.0, 1.0)
                if int8:
                    # codes are defined through the 32-bit scale and quotient
                    a = s[name][rows].float().abs().amax(-1) / 127.0
                    one = torch.where(a > 0, a, torch.ones_like(a))[..., None]
                    y = (s[name][rows].float() / one).round().double()
                    scales[name][page, :, pos % p] = a.double()
                pools[name][page, pos % p] = y
            if case["rot"]:
                q[rows] = _turn64(s["q"][rows], pos, s["freqs"],
                                  case["layout"], 1.0, 1.0)
        if int8:  # whole values, not compared as numbers
            return [q, None, None, scales["k"], scales["v"]]
        return [q, pools["k"], pools["v"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    n = s["q"].shape[0]
    out = torch.zeros((n, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((hq, n), -math.inf, dtype=torch.float64, device="cuda")
    for b, x in enumerate(lens):
        m = cu[b + 1] - cu[b]
        if m == 0 or x == 0:
            continue
        ids = torch.tensor(table[b][:-(-x // p)], device="cuda")
        kv = {}
        for name in "kv":
            y = s[name + "_pages"][ids].double()
            if case["kv"] == "int8":
                y = y * s[name + "_scale"][ids].double().transpose(1, 2)[..., None]
            kv[name] = y.flatten(0, 1)[:x]
        seen = torch.full((m,), x, device="cuda")
        if case["causal"]:
            seen = torch.arange(x - m + 1, x + 1, device="cuda")
        hidden = torch.arange(x, device="cuda")[None] >= seen[:, None]
        for h in range(hq):
            g = h // (hq // hkv)
            a = s["q"][cu[b]:cu[b + 1], h].double() @ kv["k"][:, g].t()
            a = (a / math.sqrt(d)).masked_fill(hidden, -math.inf)
            z = torch.logsumexp(a, -1)
            lse[h, cu[b]:cu[b + 1]] = z
            out[cu[b]:cu[b + 1], h] = torch.nan_to_num(
                torch.exp(a - z[:, None])) @ kv["v"][:, g]
    return [out, lse]
