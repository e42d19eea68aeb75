"""GPU cases of the paged-cache calls beyond the shapes of test_paged_gpu.py:
idle sequences of a decode batch, V scales of any size and sign, bad pages
that some rows do not reach, and the like."""
import math

import pytest

torch = pytest.importorskip("torch")

import prefill_blockwise_int8_b200 as tm
from oracle import paged as oracle
from test_paged_gpu import BAD_PAGES, BAD_SEQLENS, Cache, _check_attn, _gen

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# idle sequences (no new tokens, keys in the cache)
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["same", "int8"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,lens,hq,hkv", [
    ([1, 0], [4096, 2000], 32, 8),        # last, step kernel
    ([0, 1], [2000, 4096], 32, 8),        # first
    ([1, 0], [1000, 2000], 8, 8),         # more idle keys than active ones
    ([0, 40], [3000, 700], 8, 2),         # chunk kernel
    ([40, 0], [700, 3000], 8, 2),
    ([0] * 33 + [1] + [0] * 33 + [2], [300] * 33 + [7] + [300] * 33 + [210], 4, 1),
    ([0] * 33 + [1] + [0] * 33 + [50], [300] * 33 + [7] + [300] * 33 + [210], 4, 1),
])
def test_attn_paged_idle_sequences(new, lens, hq, hkv, causal, kv):
    c = Cache(lens, new, hkv, 64, 32, torch.float16, kv == "int8",
              seed=len(lens))
    q = torch.randn((c.cu[-1] + 1, hq, 64), generator=_gen(61)).half()
    _check_attn(c, q, causal, pad=1)


@pytest.mark.parametrize("most", [1, 64])
def test_attn_paged_nobody_active(most):
    c = Cache([100, 2000], [0, 0], 2, 64, 16, torch.float16, False)
    k, v, table, cu, lens, _ = c.device()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((5, 4, 64), 7.0, dtype=torch.float16, device="cuda")
    q = torch.randn((5, 4, 64), generator=_gen(62)).half().cuda()
    tm.tilemix_attn_paged(q, k, v, table, cu, lens, most, 2000, out=out,
                          status=status)
    assert int(status.item()) == 0 and (out == 7).all()


# ---------------------------------------------------------------------------
# V scales of any size and sign (an INT8 value is code * scale, exactly)
# ---------------------------------------------------------------------------

def _v_scales(kind, shape, pos, gen):
    """Scales [keys, heads] of one sequence's keys at positions pos."""
    x = torch.rand(shape, generator=gen) + 0.5
    sign = torch.where(torch.rand(shape, generator=gen) < 0.5, -1.0, 1.0)
    if kind == "mixed":
        return x * sign
    if kind == "cancel":   # signed sums of weights nearly vanish
        return 0.7 * (1 + 1e-5 * x) * torch.where(pos % 2 == 0, 1.0, -1.0)[:, None]
    if kind == "negative":
        return -x
    if kind == "rising":   # the reference is raised again and again
        return x * sign * 2.0 ** (pos[:, None] / 16.0 - 44)
    if kind == "falling":  # tiny beside the first
        return x * 2.0 ** (6 - pos[:, None] / 40.0)
    # nothing but zeros, then some
    return torch.where((pos // 100 % 2 == 0)[:, None], torch.zeros(()), x * sign)


@pytest.mark.parametrize("kind", ["mixed", "cancel", "negative", "rising",
                                  "falling", "zeros"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("new,d", [(1, 128), (5, 64), (40, 128), (200, 64)])
def test_attn_paged_v_scales_of_any_size_and_sign(new, d, dtype, kind):
    # one token and 20 rows: step kernel; more: chunk kernel
    c = Cache([700, 301], [new, new], 2, d, 32, dtype, True, seed=new)
    g = _gen(71)
    for b, n in enumerate(c.lens):
        pos = torch.arange(n)
        ids = c.table[b].long()[pos // 32]
        c.vs[ids, :, pos % 32] = _v_scales(kind, (n, 2), pos, g)
    if kind == "cancel":
        c.k.zero_()        # all keys weigh the same
    q = torch.randn((2 * new, 8, d), generator=_gen(72)).to(dtype)
    k, v, table, cu, lens, sc = c.device()
    out = tm.tilemix_attn_paged(q.cuda(), k, v, table, cu, lens, new, 700, **sc)
    args = (c.table, c.cu, c.lens)
    want, _, tol = oracle.attn(q, c.k, c.v, *args, k_scale=c.ks, v_scale=c.vs)
    # weights are rounded to fp16, and O is multiplied by the ratio of their
    # sums before and after: each off by at most 2^-11 of sum_j p_j |v_j|, of
    # which `tol` counts the first
    size, _, _ = oracle.attn(q, c.k, c.v.short().abs(), *args, k_scale=c.ks,
                             v_scale=c.vs.abs())
    err = (out.cpu().double() - want).abs()
    assert (err <= tol + 2.0 ** -11 * size).all(), (err / (tol + 2.0 ** -11 * size)).max()


# ---------------------------------------------------------------------------
# bad pages
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["same", "int8"])
def test_attn_paged_bad_pages_before_many_short_segments(kv):
    # every 12th sequence fills both query tiles of a block and shows a bad
    # page; the short ones behind it, 8 and more in the same block, use one
    # tile only and run ahead of the other
    batch = 1900
    new = [200 if b % 12 == 0 else 20 for b in range(batch)]
    c = Cache([n + 16 for n in new], new, 1, 64, 32, torch.float16,
              kv == "int8", seed=81)
    q = torch.randn((c.cu[-1], 1, 64), generator=_gen(82)).half().cuda()
    k, v, table, cu, lens, sc = c.device()
    call = lambda t, **kw: tm.tilemix_attn_paged(q, k, v, t, cu, lens, 200, 216,
                                                 **sc, **kw)
    good = call(table)
    broken = table.clone()
    broken[::12, 0] = 1 << 20
    out = torch.full_like(good, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(broken, out=out, status=status)
    assert int(status.item()) == BAD_PAGES
    hit = torch.zeros(c.cu[-1], dtype=torch.bool)
    for b in range(0, batch, 12):
        hit[c.cu[b]:c.cu[b + 1]] = True
    hit = hit.cuda()
    assert torch.equal(out[~hit], good[~hit]) and torch.isfinite(good).all()
    assert (out[hit] == 7).all()


@pytest.mark.parametrize("kv", ["same", "int8"])
@pytest.mark.parametrize("new,lens,page,bad", [
    (16, [600, 300], 16, {0: [37], 1: [18, 17]}),    # step kernel
    (2, [97, 5985], 32, {0: [3], 1: [187]}),         # over several blocks
    (100, [600, 300], 16, {0: [36, 33], 1: [14]}),   # chunk kernel
    (300, [1000, 6000], 64, {0: [12], 1: [91, 90]}),
    (300, [700, 290], 128, {0: [4], 1: [1]}),        # rows without keys
])
def test_attn_paged_rows_below_a_bad_page(new, lens, page, bad, kv):
    # causal rows that see no key of a bad page are computed, the rest keep
    # their outputs
    c = Cache(lens, [new] * 2, 1, 64, page, torch.float16, kv == "int8", seed=91)
    q = torch.randn((2 * new, 1, 64), generator=_gen(92)).half()
    k, v, table, cu, ln, sc = c.device()
    limit = torch.zeros(2 * new, dtype=torch.long)   # keys of each row
    first = torch.zeros(2 * new, dtype=torch.long)   # first bad key
    for b, n in enumerate(lens):
        for x in bad[b]:
            table[b, x] = -5 if x % 2 else 1 << 29
        limit[b * new:(b + 1) * new] = torch.arange(n - new + 1, n + 1)
        first[b * new:(b + 1) * new] = min(bad[b]) * page
    hit = limit > first
    assert hit.any() and (~hit).any()
    out = torch.full((2 * new, 1, 64), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((1, 2 * new), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tm.tilemix_attn_paged(q.cuda(), k, v, table, cu, ln, new, max(lens), out=out,
                          lse=lse, status=status, **sc)
    assert int(status.item()) == BAD_PAGES
    want, wl, tol = oracle.attn(q, c.k, c.v, c.table, c.cu, c.lens,
                                k_scale=c.ks, v_scale=c.vs)
    out, lse = out.cpu().double(), lse.cpu().double()
    assert (out[hit] == 7).all() and (lse[:, hit] == 7).all()
    assert ((out - want).abs()[~hit] <= tol[~hit]).all()
    seen = ~hit & ~torch.isinf(wl[0])
    assert ((lse - wl).abs()[:, seen] <= 2e-5 * (1 + wl[:, seen].abs())).all()
    assert torch.isinf(lse[:, ~hit & ~seen]).all()


# ---------------------------------------------------------------------------
# a wait that runs out
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv,new,n", [("same", 1, 700), ("int8", 1, 700),
                                      ("same", 40, 100), ("same", 40, 5000),
                                      ("int8", 40, 100), ("int8", 40, 5000)])
def test_attn_paged_expired_wait_reports_timeout(kv, new, n):
    # a first tile's barrier never completes: its bounded wait expires (2 s),
    # every copy in flight lands, rows of the blocks that gave up are not
    # written, and the next call on the same context and workspace is right.
    # With 100 keys the loads have all been issued when the wait runs out.
    c = Cache([n, n], [new, new], 1, 64, 64, torch.float16, kv == "int8", seed=5)
    q = torch.randn((2 * new, 2, 64), generator=_gen(6)).half()
    k, v, table, cu, lens, sc = c.device()
    ws = torch.empty(tm.tilemix_attn_paged_workspace_bytes(new, 2, 1, 64),
                     dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((2 * new, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    tm.tilemix_attn_paged(q.cuda(), k, v, table, cu, lens, new, n, out=out,
                          workspace=ws, status=status, test_expire_wait=True, **sc)
    end.record()
    torch.cuda.synchronize()
    assert int(status.item()) == 4 and start.elapsed_time(end) < 30e3
    assert (out == 7).all()
    _check_attn(c, q, True, workspace=ws)


# ---------------------------------------------------------------------------
# appending
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rot", [0, 64])
@pytest.mark.parametrize("new", [3, 1100])   # one and 16 tokens a block
def test_append_int8_keeps_non_finite_rows_visible(new, rot, dtype):
    c = Cache([new + 9], [new], 2, 64, 32, dtype, True, seed=3)
    x = torch.randn((new, 4, 64), generator=_gen(4)).to(dtype)
    x[0, 0, 5], x[1, 1, 60] = math.nan, math.inf
    x[1, 2, 0], x[2, 3, 63] = -math.inf, math.nan
    x[2, 0, 1], x[2, 0, 2] = math.inf, math.nan
    k, v, table, cu, lens, sc = c.device()
    freqs = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)],
                         dtype=torch.float64).cuda() if rot else None
    tm.tilemix_paged_append(x[:, :2].cuda(), x[:, 2:].cuda(), table, cu, lens,
                            k, v, freqs=freqs, **sc)
    rows = x.clone()
    if rot:
        pos = torch.arange(9, new + 9, dtype=torch.int32).cuda()
        rows[:, :2] = tm.tilemix_rope(x[:, :2].cuda(), None, pos, freqs)[0].cpu()
    for t, b, p, pid, slot in oracle.places(c.cu, c.lens, c.table.tolist(), 32):
        codes = torch.cat((k[pid, slot], v[pid, slot])).cpu()
        scale = torch.cat((sc["k_scale"][pid, :, slot],
                           sc["v_scale"][pid, :, slot])).cpu()
        top = rows[t].float().abs().amax(-1)   # NaN where the row has one
        bad = ~torch.isfinite(top)
        assert torch.equal(torch.isnan(scale), bad)
        want, ws = oracle.quantised(rows[t])
        assert torch.equal(codes[~bad], want[~bad])
        assert torch.equal(scale[~bad], ws[~bad])
        if t == 6:
            break


@pytest.mark.parametrize("kv", ["same", "int8"])
@pytest.mark.parametrize("pad", [0, 1200])   # one and several tokens a block
def test_append_reports_every_bad_sequence(kv, pad):
    # also where no token is placed by it: a decreasing end, idle sequences
    c = Cache([40, 50, 30], [6, 4, 0], 2, 64, 16, torch.float16, kv == "int8")
    x = torch.randn((10 + pad, 2, 64), generator=_gen(7)).half().cuda()
    _, _, table, cu, lens, _ = c.device()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()
    for bad_cu, bad_lens, want in [
            ([0, 6, 10, 10], [40, 50, 30], 0),
            ([0, 10, 4, 4], [40, 50, 30], BAD_SEQLENS),
            ([0, 6, 10, 9], [40, 50, 30], BAD_SEQLENS),
            ([0, 6, 10, 10], [40, 50, -1], BAD_SEQLENS),
            ([0, 6, 10, 10], [40, 50, 1 << 20], BAD_SEQLENS),
            ([0, 6, 10, 11 + pad], [40, 50, 30], BAD_SEQLENS),
            ([-1, 6, 10, 10], [40, 50, 30], BAD_SEQLENS)]:
        k, v, _, _, _, sc = c.device()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tm.tilemix_paged_append(x, x, table, i32(bad_cu), i32(bad_lens), k, v,
                                status=status, **sc)
        assert int(status.item()) == want, (bad_cu, bad_lens)


@pytest.mark.parametrize("kv", ["same", "int8"])
@pytest.mark.parametrize("new", [3, 600])
def test_rows_before_the_first_sequence_are_padding(new, kv):
    c = Cache([new + 7, new + 30], [new, new], 2, 64, 32, torch.float16,
              kv == "int8", poison=False)
    x = torch.randn((2 * new + 5, 8, 64), generator=_gen(8)).half().cuda()
    k, v, table, cu, lens, sc = c.device()
    k2, v2, _, _, _, sc2 = c.device()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = torch.tensor([10000.0 ** (-i / 16.0) for i in range(16)],
                     dtype=torch.float64).cuda()
    qo = torch.full((2 * new + 5, 4, 64), 7.0, dtype=torch.float16, device="cuda")
    args = dict(freqs=f, status=status)
    tm.tilemix_paged_append(x[:, :2], x[:, 2:4], table, cu + 5, lens, k, v,
                            q=x[:, 4:], q_out=qo, **args, **sc)
    want = tm.tilemix_paged_append(x[5:, :2], x[5:, 2:4], table, cu, lens, k2, v2,
                                   q=x[5:, 4:], **args, **sc2)
    assert int(status.item()) == 0
    assert torch.equal(k, k2) and torch.equal(v, v2)
    assert (qo[:5] == 7).all() and torch.equal(qo[5:], want)
    out = torch.full_like(qo, 7.0)
    tm.tilemix_attn_paged(qo, k, v, table, cu + 5, lens, new, new + 30, out=out,
                          status=status, **sc)
    ref = tm.tilemix_attn_paged(want, k, v, table, cu, lens, new, new + 30, **sc)
    assert int(status.item()) == 0
    assert (out[:5] == 7).all() and torch.equal(out[5:], ref)


def test_attn_paged_bounds_beyond_32_bits_are_refused():
    c = Cache([30], [1], 1, 64, 16, torch.float16, False)
    k, v, table, cu, lens, _ = c.device()
    q = torch.zeros((1, 1, 64), dtype=torch.float16, device="cuda")
    for a, b in ((1 << 31, 30), (1, 1 << 31), ((1 << 32) + 1, 30)):
        with pytest.raises(ValueError, match="2\\^31"):
            tm.tilemix_attn_paged(q, k, v, table, cu, lens, a, b)
    with pytest.raises(tm.TilemixError):
        tm.tilemix_attn_paged(q, k, v, table, cu, lens, 1 << 30 | 1, 30)


# ---------------------------------------------------------------------------
# the rotation's gradient
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_rope_gradient_is_recorded(layout, dtype):
    g = _gen(15)
    qkv = torch.randn((9, 8, 64), generator=g).to(dtype).cuda().requires_grad_()
    pos = torch.tensor([0, 1, 5, 77, 300, 4096, 9, 9, 100000], dtype=torch.int32)
    f = torch.tensor([10000.0 ** (-i / 16.0) for i in range(16)],
                     dtype=torch.float64)
    go = torch.randn((9, 6, 64), generator=g).to(dtype)
    kw = dict(layout=layout, attn_factor=1.25)
    q, k = tm.tilemix_rope(qkv[:, :4], qkv[:, 4:6], pos.cuda(), f.cuda(), **kw)
    plain, plain_k = tm.tilemix_rope(qkv.detach()[:, :4], qkv.detach()[:, 4:6],
                                     pos.cuda(), f.cuda(), **kw)
    assert torch.equal(q, plain) and torch.equal(k, plain_k)
    assert q.requires_grad and k.requires_grad and not plain.requires_grad
    (gx,) = torch.autograd.grad([q, k], [qkv], [go[:, :4].cuda(), go[:, 4:].cuda()],
                                retain_graph=True)
    want = oracle.rope(go, pos, f, layout, 1.25, True)
    half = torch.finfo(dtype).eps / 2
    # the rounded value, and fp32 cosines and sines of angles that are off by
    # 2 pi 2^-26 and 3 2^-53 of up to 1e5 radians
    tol = half * want.abs() + oracle.rope_bound(go, f, layout, 1.25, 1.2e-7) + 2.0 ** -25
    assert ((gx[:, :6].cpu().double() - want).abs() <= tol).all()
    assert (gx[:, 6:] == 0).all()
    # one output only, expanded and misplaced gradients
    (gq,) = torch.autograd.grad(q, [qkv], go[:, :4].cuda(), retain_graph=True)
    assert torch.equal(gq[:, :4], gx[:, :4]) and (gq[:, 4:] == 0).all()
    (gk,) = torch.autograd.grad(k, [qkv], go[:, 4:].cuda(), retain_graph=True)
    assert torch.equal(gk[:, 4:6], gx[:, 4:6]) and (gk[:, :4] == 0).all()
    ones = torch.ones_like(q)
    (a,) = torch.autograd.grad(q, [qkv], ones, retain_graph=True)
    (b,) = torch.autograd.grad(q.sum(), [qkv], retain_graph=True)
    assert torch.equal(a, b)
    odd = torch.randn((9 * 4 * 64 + 1,), generator=g).to(dtype).cuda()[1:].view(9, 4, 64)
    (a,) = torch.autograd.grad(q, [qkv], odd, retain_graph=True)
    (b,) = torch.autograd.grad(q, [qkv], odd.clone(), retain_graph=True)
    assert torch.equal(a, b)
    # the gradient's own gradient is the rotation
    w = go[:, :4].cuda().requires_grad_()
    (d,) = torch.autograd.grad(q, [qkv], w, create_graph=True)
    (ww,) = torch.autograd.grad(d[:, :4], [w], qkv.detach()[:, :4])
    assert torch.equal(ww, plain)


def test_rope_gradient_without_k_streams_and_refusals():
    x = torch.randn((5, 2, 64), generator=_gen(16)).half().cuda().requires_grad_()
    pos = torch.arange(5, dtype=torch.int32).cuda()
    f = torch.tensor([10000.0 ** (-i / 32.0) for i in range(32)],
                     dtype=torch.float64).cuda()
    y, none = tm.tilemix_rope(x, None, pos, f)
    assert none is None
    y.backward(torch.ones_like(y))
    want, _ = tm.tilemix_rope(torch.ones_like(y).detach(), None, pos, f, inverse=True)
    assert torch.equal(x.grad, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z, _ = tm.tilemix_rope(x, None, pos, f, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    (gz,) = torch.autograd.grad(z, [x], torch.ones_like(z))
    torch.cuda.synchronize()
    assert torch.equal(z, y) and torch.equal(gz, want)
    # k alone needs one
    q = x.detach()
    yq, yk = tm.tilemix_rope(q, x, pos, f)
    (gk,) = torch.autograd.grad(yk, [x], torch.ones_like(yk))
    assert torch.equal(gk, want) and torch.equal(yq, y)
    with pytest.raises(ValueError, match="autograd"):
        tm.tilemix_rope(x, None, pos, f, q_out=torch.empty_like(q))
    with torch.no_grad():
        out = torch.empty_like(q)
        tm.tilemix_rope(x, None, pos, f, q_out=out)
    assert torch.equal(out, y) and not out.requires_grad


# ---------------------------------------------------------------------------
# together with the prefill, and mixed batches
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["same", "int8"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
def test_prefill_attention_then_paged_decode(d, page, kv):
    """A prompt goes through the prefill attention (all FP16) while its K and V
    enter the pages; the paged attention of the same tokens agrees, and decoded
    tokens continue over the pages."""
    int8 = kv == "int8"
    hq, hkv, n = 4, 2, [200, 131]
    x = [torch.randn((m + 2, hq + 2 * hkv, d), generator=_gen(17 + m)).half()
         for m in n]
    pages = sum(-(-(m + 2) // page) for m in n)
    kp = torch.zeros((pages, page, hkv, d), device="cuda",
                     dtype=torch.int8 if int8 else torch.float16)
    vp = torch.zeros_like(kp)
    sc = dict(k_scale=torch.zeros((pages, hkv, page), device="cuda"),
              v_scale=torch.zeros((pages, hkv, page), device="cuda")) if int8 else {}
    first = -(-(n[0] + 2) // page)
    order = list(range(pages))[::-1]
    table = torch.tensor([order[:first], order[first:] + [-1] * (2 * first - pages)],
                         dtype=torch.int32).cuda()
    freqs, _ = tm.tilemix_rope_frequencies(d, 10000.0, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()
    rot, outs = [[], []], [[], []]
    for step, (a, b) in enumerate([(0, n), (n, [m + 1 for m in n]),
                                   ([m + 1 for m in n], [m + 2 for m in n])]):
        a = [0, 0] if a == 0 else a
        y = torch.cat([x[s][a[s]:b[s]] for s in range(2)]).cuda()
        new = [b[s] - a[s] for s in range(2)]
        cu, ln = i32([0, new[0], sum(new)]), i32(b)
        q = tm.tilemix_paged_append(
            y[:, hq:hq + hkv], y[:, hq + hkv:], table, cu, ln, kp, vp,
            q=y[:, :hq], freqs=freqs, **sc)
        o = tm.tilemix_attn_paged(q, kp, vp, table, cu, ln, max(new), max(b), **sc)
        if step == 0:
            pos = torch.cat([torch.arange(m) for m in n]).int().cuda()
            _, kr = tm.tilemix_rope(y[:, :hq], y[:, hq:hq + hkv], pos, freqs)
            pre = tm.tilemix_attn_prefill(
                q, kr, y[:, hq + hkv:].contiguous(), cu, max(n), fp16_only=True)
            if not int8:
                assert (pre.float() - o.float()).abs().max() <= 3e-3
        for s, r in ((0, slice(0, new[0])), (1, slice(new[0], sum(new)))):
            rot[s].append(q[r].cpu())
            outs[s].append((o if int8 or step else pre)[r].cpu())
    host = {name: t.cpu() for name, t in sc.items()}
    for s in range(2):
        m = n[s] + 2
        want, _, tol = oracle.attn(torch.cat(rot[s]), kp.cpu(), vp.cpu(),
                                   [table[s].tolist()], [0, m], [m], **host)
        err = (torch.cat(outs[s]).double() - want).abs()
        # (the prefill's rows to its own tolerance)
        assert (err[n[s]:] <= tol[n[s]:]).all()
        assert (err[:n[s]] <= (tol[:n[s]] if int8 else 3e-3)).all()


@pytest.mark.parametrize("kv", ["same", "int8"])
def test_attn_paged_one_chunk_among_single_tokens(kv):
    new = [1] * 20 + [300] + [1] * 27
    lens = [1 + 37 * b % 900 for b in range(48)]
    lens[20] = 1400
    c = Cache(lens, new, 2, 64, 32, torch.float16, kv == "int8", seed=18)
    q = torch.randn((c.cu[-1] + 2, 4, 64), generator=_gen(19)).half()
    _check_attn(c, q, True, pad=2)


def test_attn_paged_repeats_exactly_on_other_memory():
    # the same call again, on other memory: bit for bit the same
    for new, n, hq, hkv, kv in ((1, 8191, 8, 8, True), (1, 4096, 8, 2, False),
                                (5, 3000, 28, 4, False), (700, 2000, 6, 2, True),
                                (700, 2000, 6, 2, False)):
        c = Cache([n, n // 3], [new, min(new, n // 3)], hkv, 128, 64,
                  torch.float16, kv, seed=n)
        q = torch.randn((c.cu[-1], hq, 128), generator=_gen(n + 1)).half().cuda()
        first = None
        for _ in range(3):
            k, v, table, cu, lens, sc = c.device()
            keep = torch.full((1 << 22,), 3.0, device="cuda")
            lse = torch.empty((hq, c.cu[-1]), device="cuda")
            out = tm.tilemix_attn_paged(q, k, v, table, cu, lens, new, n, lse=lse,
                                        **sc)
            first = first or (out, lse)
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
            del keep


@pytest.mark.parametrize("new", [1, 40])
def test_strides_of_axes_of_one_do_not_matter(new):
    # one KV head: token-major K and head-major V are the same layout
    c = Cache([90], [new], 1, 64, 16, torch.float16, False, seed=20)
    k, v, table, cu, lens, _ = c.device()
    v = v.transpose(1, 2).contiguous().transpose(1, 2)
    n, page, _, d = v.shape
    v = v.as_strided((n, page, 1, d), (page * d, d, page * d, 1))
    assert k.stride() != v.stride()
    q = torch.randn((new, 4, 64), generator=_gen(21)).half()
    _check_attn(c, q, True, device=(k, v, table, cu, lens, {}))
    with pytest.raises(ValueError, match="strides"):
        wide = torch.zeros((n, page, 1, 2 * d), dtype=v.dtype, device="cuda")
        tm.tilemix_attn_paged(q.cuda(), k, wide[..., :d], table, cu, lens, new, 90)


@pytest.mark.parametrize("kv", ["same", "int8"])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_a_captured_serving_step_replays_over_a_growing_cache(new, kv):
    """Append and attention in one captured graph: lengths move on the device,
    every replay's tokens equal causal attention over all that was appended."""
    int8 = kv == "int8"
    hq, hkv, d, page, steps = 16, 2, 64, 16, 4
    start = [30, 7]
    pages = 30
    kp = torch.zeros((pages, page, hkv, d), device="cuda",
                     dtype=torch.int8 if int8 else torch.bfloat16)
    vp = torch.zeros_like(kp)
    sc = dict(k_scale=torch.zeros((pages, hkv, page), device="cuda"),
              v_scale=torch.zeros((pages, hkv, page), device="cuda")) if int8 else {}
    table = torch.randperm(pages, generator=_gen(31)).int().view(2, 15).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()
    freqs, _ = tm.tilemix_rope_frequencies(d, 10000.0, device="cuda")
    heads = hq + 2 * hkv
    old = torch.randn((sum(start), heads, d), generator=_gen(32)).bfloat16().cuda()
    lens = i32(start)
    qs = [[], []]
    q0 = tm.tilemix_paged_append(old[:, hq:hq + hkv], old[:, hq + hkv:], table,
                                 i32([0, start[0], sum(start)]), lens, kp, vp,
                                 q=old[:, :hq], freqs=freqs, **sc)
    qs[0].append(q0[:start[0]].cpu())
    qs[1].append(q0[start[0]:].cpu())
    cu = i32([0, new, 2 * new])
    x = torch.zeros((2 * new, heads, d), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((2 * new, hq, d), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(tm.tilemix_attn_paged_workspace_bytes(new, hq, hkv, d),
                     dtype=torch.uint8, device="cuda")
    most = max(start) + steps * new

    def step():
        lens.add_(new)
        tm.tilemix_paged_append(x[:, hq:hq + hkv], x[:, hq + hkv:], table, cu, lens,
                                kp, vp, q=x[:, :hq], q_out=q, freqs=freqs, **sc)
        tm.tilemix_attn_paged(q, kp, vp, table, cu, lens, new, most, out=out,
                              workspace=ws, **sc)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    outs = [[], []]
    for s in range(steps):
        x.copy_(torch.randn(x.shape, generator=_gen(40 + s)))
        graph.replay()
        for b in range(2):
            qs[b].append(q[b * new:(b + 1) * new].cpu())
            outs[b].append(out[b * new:(b + 1) * new].cpu())
    assert lens.tolist() == [n + steps * new for n in start]
    for b in range(2):
        n = start[b] + steps * new
        want, _, tol = oracle.attn(
            torch.cat(qs[b]), kp.cpu(), vp.cpu(), [table[b].tolist()], [0, n], [n],
            **{name: t.cpu() for name, t in sc.items()})
        err = (torch.cat(outs[b]).double() - want[start[b]:]).abs()
        assert (err <= tol[start[b]:]).all()


@pytest.mark.parametrize("kv", ["same", "int8"])
@pytest.mark.parametrize("new", [1, 50])
def test_sequences_that_share_pages(new, kv):
    # one prompt's pages in every row of the table, lengths of their own
    c = Cache([500], [new], 2, 64, 16, torch.float16, kv == "int8", seed=51)
    c.table = c.table.repeat(3, 1)
    c.lens, c.new = [500, 77 + new, 320], [new] * 3
    c.cu = [0, new, 2 * new, 3 * new]
    q = torch.randn((3 * new, 8, 64), generator=_gen(52)).half()
    _check_attn(c, q, True)


@pytest.mark.parametrize("kv", ["same", "int8"])
def test_two_caches_grow_on_two_streams_at_once(kv):
    caches = [Cache([900, 40], [600, 40], 2, 128, 32, torch.float16, kv == "int8",
                    seed=60 + i, poison=False) for i in range(2)]
    x = torch.randn((640, 12, 128), generator=_gen(61)).half().cuda()
    f = torch.tensor([10000.0 ** (-i / 64.0) for i in range(64)],
                     dtype=torch.float64).cuda()

    def step(dev, stream):
        k, v, table, cu, lens, sc = dev
        q = tm.tilemix_paged_append(x[:, 8:10], x[:, 10:], table, cu, lens, k, v,
                                    q=x[:, :8], freqs=f, stream=stream, **sc)
        return q, tm.tilemix_attn_paged(q, k, v, table, cu, lens, 600, 900,
                                        stream=stream, **sc)

    plain = [c.device() for c in caches]
    want = [step(dev, None) for dev in plain]
    both = [c.device() for c in caches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):  # appending the same tokens again changes nothing
        for i in range(2):
            got[i] = step(both[i], streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(want[i], got[i]):
            assert torch.equal(a, b)
        for a, b in zip(plain[i][:2], both[i][:2]):
            assert torch.equal(a, b)
        for name, t in plain[i][5].items():
            assert torch.equal(t, both[i][5][name])
