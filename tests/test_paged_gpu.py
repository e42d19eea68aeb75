"""GPU parity of the rotary and paged-cache calls against their 64-bit oracle
(oracle/paged.py): sizes and masks where they can go wrong, strides, streams,
graphs, bad pages, and a serving loop that uses all of them together."""
import math

import pytest

torch = pytest.importorskip("torch")

import prefill_blockwise_int8_b200 as tm
from oracle import paged as oracle

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
BAD_SEQLENS, BAD_PAGES = 5, 7


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _freqs(rot, base=10000.0):
    return torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)],
                        dtype=torch.float64)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,hq,hkv,d,rot", [
    (1, 1, 1, 64, 64), (3, 5, 1, 128, 128), (7, 4, 2, 128, 32),
    (2, 3, 3, 80, 16), (5, 2, 1, 96, 96), (1100, 2, 1, 64, 32),
    (4, 33, 8, 256, 256), (2, 1, 1, 16, 16), (9, 7, 1, 112, 64)])
def test_rope(dtype, layout, tokens, hq, hkv, d, rot):
    t = TYPES[dtype]
    g = _gen(tokens * 31 + d)
    qkv = torch.randn((tokens, hq + 2 * hkv, d), generator=g).to(t)
    pos = torch.randint(-5, 1 << 20, (tokens,), generator=g, dtype=torch.int32)
    pos[0] = (1 << 31) - 1
    freqs = _freqs(rot)
    dev = qkv.cuda()
    for inverse, factor in ((False, 1.0), (True, 1.25)):
        q, k = tm.tilemix_rope(dev[:, :hq], dev[:, hq:hq + hkv], pos.cuda(),
                               freqs.cuda(), layout=layout, inverse=inverse,
                               attn_factor=factor)
        for got, x in ((q, qkv[:, :hq]), (k, qkv[:, hq:hq + hkv])):
            want = oracle.rope(x, pos, freqs, layout, factor, inverse)
            # the angle: 2^-26 turns for the fp32 remainder, 3 * 2^-53 of the
            # turns (the last position: 2^31 / 2 pi) for the products
            angle = 2 * math.pi * (2.0 ** -26 + 2.0 ** 31 / 6.28 * 3 * 2.0 ** -53)
            tol = HALF_STEP[t] * want.abs() + 2.0 ** -25 + \
                1.01 * oracle.rope_bound(x, freqs, layout, factor, angle)
            assert ((got.cpu().double() - want).abs() <= tol).all()
            assert torch.equal(got[..., rot:].cpu(), x[..., rot:])


def test_rope_in_place_without_k_and_empty():
    g = _gen(3)
    x = torch.randn((6, 4, 64), generator=g).half().cuda()
    pos = torch.arange(6, dtype=torch.int32).cuda()
    f = _freqs(64).cuda()
    want, none = tm.tilemix_rope(x, None, pos, f)
    assert none is None
    y = x.clone()
    got, _ = tm.tilemix_rope(y, None, pos, f, q_out=y)
    assert got is y and torch.equal(y, want)
    # head-major storage on both sides
    xt = x.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty((4, 6, 64), dtype=x.dtype, device="cuda").transpose(0, 1)
    got, _ = tm.tilemix_rope(xt, None, pos, f, q_out=out)
    assert torch.equal(got, want)
    e, ek = tm.tilemix_rope(x[:0], x[:0, :1], pos[:0], f)
    assert e.shape == (0, 4, 64) and ek.shape == (0, 1, 64)


def test_rope_inverse_is_the_gradient():
    # <g, R x> = <R^T g, x> with R^T the inverse rotation, and by differences
    g = _gen(4)
    t, h, d = 5, 3, 64
    x, go = (torch.randn((t, h, d), generator=g).half() for _ in range(2))
    pos = torch.tensor([0, 1, 77, 4096, 100000], dtype=torch.int32)
    f = _freqs(48)
    for layout in ("half", "interleaved"):
        gx, _ = tm.tilemix_rope(go.cuda(), None, pos.cuda(), f.cuda(),
                                layout=layout, inverse=True, attn_factor=1.5)
        want = oracle.rope(go, pos, f, layout, 1.5, True)
        assert ((gx.cpu().double() - want).abs() <=
                2.0 ** -10 * want.abs() + 1e-5).all()
        step = torch.randn((t, h, d), generator=g).double()
        diff = (oracle.rope(x.double() + step, pos, f, layout, 1.5) -
                oracle.rope(x.double() - step, pos, f, layout, 1.5)) / 2
        lhs = (go.double() * diff).sum()
        rhs = (want * step).sum()
        assert abs(lhs - rhs) <= 1e-9 * (go.double() * diff).abs().sum()


def test_rope_backward_captured_while_eager_results_live():
    x = torch.randn((33, 4, 128), generator=_gen(5)).bfloat16().cuda()
    pos = torch.arange(33, dtype=torch.int32).cuda()
    f = _freqs(128).cuda()
    y, _ = tm.tilemix_rope(x, None, pos, f)
    back, _ = tm.tilemix_rope(y, None, pos, f, inverse=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, _ = tm.tilemix_rope(x, None, pos, f)
        back2, _ = tm.tilemix_rope(y2, None, pos, f, inverse=True)
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    # halving is exact, and so is the rotation's image of it
    assert torch.equal(y2, y * 0.5) and torch.equal(back2, back * 0.5)


# ---------------------------------------------------------------------------
# a cache
# ---------------------------------------------------------------------------

class Cache:
    """Pages of random contents (or NaN / extreme codes in slots that no
    sequence owns), a shuffled page table with unused entries of -7."""

    def __init__(self, lens, new, hkv, d, page, dtype, int8, seed=0,
                 layout="token", poison=True, spare=2):
        g = _gen(seed)
        self.lens, self.new, self.page, self.int8 = lens, new, page, int8
        self.cu = [0]
        for m in new:
            self.cu.append(self.cu[-1] + m)
        counts = [-(-n // page) for n in lens]
        total = sum(counts) + spare
        order = torch.randperm(total, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), max(1, max(counts, default=0)) + 1),
                                -7, dtype=torch.int32)
        at = 0
        live = torch.zeros((total, page), dtype=torch.bool)
        for b, c in enumerate(counts):
            ids = order[at:at + c]
            self.table[b, :c] = ids
            at += c
            for i, x in enumerate(ids.tolist()):
                live[x, :min(page, lens[b] - i * page)] = True
        self.live = live
        shape = (total, page, hkv, d)
        k, v = (torch.randn(shape, generator=g) for _ in range(2))
        k[..., 1] *= 8
        if int8:
            self.k, self.ks = oracle.quantised(k)
            self.v, self.vs = oracle.quantised(v)
            self.ks = self.ks.transpose(1, 2).contiguous()
            self.vs = self.vs.transpose(1, 2).contiguous()
            if poison:
                dead = ~live[:, None, :].expand(total, hkv, page)
                self.ks[dead] = math.nan
                self.vs[dead] = math.inf
        else:
            self.k, self.v, self.ks, self.vs = k.to(dtype), v.to(dtype), None, None
            if poison:
                self.k[~live] = math.nan
                self.v[~live] = math.nan
        self.layout = layout

    def device(self):
        """k, v pages, table, cu, lens on the GPU; scales as keywords."""
        def pages(x):
            x = x.cuda()
            if self.layout == "head":    # [pages][heads][slots][d]
                x = x.transpose(1, 2).contiguous().transpose(1, 2)
            if self.layout == "padded":  # heads further apart
                y = torch.zeros(x.shape[:3] + (x.shape[3] + 32,),
                                dtype=x.dtype, device="cuda")
                y[..., :x.shape[3]] = x
                x = y[..., :x.shape[3]]
            return x
        kw = {}
        if self.int8:
            kw = dict(k_scale=self.ks.cuda(), v_scale=self.vs.cuda())
        i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()
        return (pages(self.k), pages(self.v), self.table.cuda(), i32(self.cu),
                i32(self.lens), kw)


def _check_attn(c, q, causal, scale=None, pad=0, device=None, **kw):
    k, v, table, cu, lens, scales = device or c.device()
    t, hq, d = q.shape
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.full((hq, t), 7.0, device="cuda")
    out = torch.full((t, hq, d), 7.0, dtype=q.dtype, device="cuda")
    tm.tilemix_attn_paged(
        q.cuda(), k, v, table, cu, lens, max(c.new, default=0),
        max(c.lens, default=0), causal=causal, softmax_scale=scale or 0.0,
        out=out, lse=lse, status=status, **scales, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    n = t - pad
    want, wl, tol = oracle.attn(
        q[:n], c.k, c.v, c.table, c.cu, c.lens, causal=causal, scale=scale,
        k_scale=c.ks, v_scale=c.vs)
    got = out.cpu().double()
    err = (got[:n] - want).abs()
    assert (err <= tol).all(), (err - tol).max()
    gl = lse.cpu().double()
    empty = torch.isinf(wl)
    assert torch.equal(torch.isinf(gl[:, :n]), empty)
    # 2 ds of a score's error at worst, 2^-20 for the sums and logarithm
    le = (gl[:, :n] - wl)[~empty].abs()
    assert (le <= 2e-5 * (1 + wl[~empty].abs())).all()
    assert (got[n:] == 7).all() and (gl[:, n:] == 7).all()
    return out, lse


SHAPES = [
    # new tokens, lengths, hq, hkv, d, page
    ([1], [1], 1, 1, 64, 16),
    ([1], [0], 2, 1, 128, 16),                 # no key at all (not causal)
    ([1, 1, 1], [1, 17, 300], 8, 2, 128, 16),
    ([1, 0, 1], [5, 9, 64], 4, 4, 64, 32),
    ([1] * 40, list(range(1, 41)), 8, 8, 128, 16),
    ([1, 1], [2049, 1000], 32, 8, 128, 128),
    ([5, 5, 5], [5, 100, 257], 28, 4, 128, 64),
    ([3, 0, 17], [50, 40, 17], 7, 1, 64, 16),
    ([33, 1], [33, 513], 6, 2, 128, 256),
    ([1], [130], 128, 1, 128, 16),
    ([2], [77], 40, 1, 64, 32),
    ([130, 64, 1], [400, 64, 9], 6, 2, 128, 32),
    ([129], [129], 2, 2, 64, 64),
    ([257, 300], [700, 300], 4, 4, 128, 16),
    ([300, 7, 140], [1024, 500, 141], 8, 1, 128, 128),
    ([513], [1500], 3, 1, 64, 32),
    ([3, 0, 2], [100, 33, 700], 16, 2, 128, 16),   # 17 to 32 packed rows
    ([1, 1], [90, 2500], 24, 1, 64, 32),           # a group above 16
    ([4], [1000], 32, 4, 64, 16),
]


@pytest.mark.parametrize("kv", ["same", "int8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_attn_paged(i, causal, dtype, kv):
    new, lens, hq, hkv, d, page = SHAPES[i]
    lens = list(lens)
    if not causal:  # an encoder's states: any length, the queries not in it
        lens = [n if n < 1000 else n - 700 for n in lens]
    elif 0 in lens:
        lens = [max(n, m) for n, m in zip(lens, new)]
    t = TYPES[dtype]
    c = Cache(lens, new, hkv, d, page, t, kv == "int8", seed=i,
              layout=("token", "head", "padded")[i % 3])
    pad = i % 3
    q = torch.randn((c.cu[-1] + pad, hq, d), generator=_gen(i + 50)).to(t)
    _check_attn(c, q, causal, pad=pad)


@pytest.mark.parametrize("kv", ["same", "int8"])
def test_attn_paged_rows_without_keys(kv):
    # fewer keys than new tokens: the first rows of the causal mask are empty
    c = Cache([3, 0, 40], [10, 4, 150], 2, 64, 16, torch.float16, kv == "int8")
    q = torch.randn((164, 6, 64), generator=_gen(9)).half()
    _check_attn(c, q, True)


@pytest.mark.parametrize("kv", ["same", "int8"])
@pytest.mark.parametrize("new", [1, 40, 300])
def test_attn_paged_strided_q_scale_and_large_scores(kv, new):
    c = Cache([500, 301], [new, new], 2, 128, 64, torch.bfloat16, kv == "int8",
              seed=new)
    qkv = torch.randn((2 * new, 12, 128), generator=_gen(11)).bfloat16()
    qkv[:, :, 1] *= 8          # scores of some hundreds
    q = qkv[:, 2:10]
    dev = qkv.cuda()[:, 2:10]
    assert not dev.is_contiguous()
    k, v, table, cu, lens, scales = c.device()
    out = tm.tilemix_attn_paged(dev, k, v, table, cu, lens, new, 500,
                                softmax_scale=0.2, **scales)
    want, _, tol = oracle.attn(q, c.k, c.v, c.table, c.cu, c.lens, scale=0.2,
                               k_scale=c.ks, v_scale=c.vs)
    assert ((out.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("kv", ["same", "int8"])
@pytest.mark.parametrize("new", [5, 200])
def test_attn_paged_non_finite_keys_reach_their_rows_only(new, kv):
    # key 400 + new - 3 is seen by the last three rows; a NaN there makes them
    # NaN, an infinity too (by the formula: inf - inf), the others stay
    c = Cache([400 + new, 300 + new], [new, new], 2, 64, 32, torch.float16,
              kv == "int8", seed=31)
    q = torch.rand((2 * new, 4, 64), generator=_gen(32)).half() + 0.1
    at = 400 + new - 3
    pid, slot = int(c.table[0, at // 32]), at % 32
    for bad in (math.nan, math.inf):
        k, v, table, cu, lens, sc = c.device()
        if kv == "int8":
            k[pid, slot] = 1  # scores of one sign
            sc["k_scale"][pid, :, slot] = bad
        else:
            k[pid, slot, :, 7] = bad
        want, wl, tol = oracle.attn(q, c.k, c.v, c.table, c.cu, c.lens,
                                    k_scale=c.ks, v_scale=c.vs)
        lse = torch.empty((4, 2 * new), device="cuda")
        out = tm.tilemix_attn_paged(q.cuda(), k, v, table, cu, lens, new,
                                    400 + new, lse=lse, **sc).cpu().double()
        hit = torch.zeros(2 * new, dtype=torch.bool)
        hit[new - 3:new] = True
        assert torch.isnan(out[hit]).all() and torch.isnan(lse.cpu()[:, hit]).all()
        assert ((out[~hit] - want[~hit]).abs() <= tol[~hit]).all()
        assert torch.isfinite(lse.cpu()[:, ~hit]).all()


@pytest.mark.parametrize("new", [1, 9])
def test_append_and_attn_paged_many_sequences(new):
    # far more sequences than a warp looks at in one step
    batch, hq, hkv, d, page = 1100, 4, 1, 64, 16
    g = _gen(41)
    lens = (torch.randint(0, 40, (batch,), generator=g) + new).tolist()
    c = Cache(lens, [new] * batch, hkv, d, page, torch.bfloat16, False, seed=42)
    x = torch.randn((batch * new, hq + 2 * hkv, d), generator=g).bfloat16()
    k, v, table, cu, ln, _ = c.device()
    dev = x.cuda()
    tm.tilemix_paged_append(dev[:, hq:hq + 1], dev[:, hq + 1:], table, cu, ln, k, v)
    for t, b, p, pid, slot in oracle.places(c.cu, lens, c.table.tolist(), page):
        c.k[pid, slot], c.v[pid, slot] = x[t, hq:hq + 1], x[t, hq + 1:]
    live = c.live
    assert torch.equal(k.cpu()[live], c.k[live])
    assert torch.equal(v.cpu()[live], c.v[live])
    out = tm.tilemix_attn_paged(dev[:, :hq], k, v, table, cu, ln, new, max(lens))
    want, _, tol = oracle.attn(x[:, :hq], c.k, c.v, c.table, c.cu, lens)
    assert ((out.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("kv", ["same", "int8"])
def test_attn_paged_blocks_that_change_between_few_and_many_rows(kv):
    # sequences of at most and of more than 128 packed rows by turns, long
    # enough that every block takes several of both: the second query tile's
    # warps sit out some of a block's segments
    batch = 36
    new = [3 if b % 2 else 130 for b in range(batch)]
    lens = [1500 + 16 * b if b % 2 else 900 + b for b in range(batch)]
    c = Cache(lens, new, 8, 64, 64, torch.float16, kv == "int8", seed=21)
    q = torch.randn((c.cu[-1], 8, 64), generator=_gen(22)).half()
    q[:, :, 1] *= 4
    k, v, table, cu, ln, sc = c.device()
    lse = torch.empty((8, c.cu[-1]), device="cuda")
    out = tm.tilemix_attn_paged(q.cuda(), k, v, table, cu, ln, 130, max(lens),
                                lse=lse, **sc)
    # one head of each sequence against the oracle
    for b in range(batch):
        h = b % 8
        kv1 = dict(k_scale=c.ks[:, h:h + 1], v_scale=c.vs[:, h:h + 1]) \
            if kv == "int8" else {}
        rows = slice(c.cu[b], c.cu[b + 1])
        want, wl, tol = oracle.attn(q[rows, h:h + 1], c.k[:, :, h:h + 1],
                                    c.v[:, :, h:h + 1], [c.table[b]],
                                    [0, new[b]], [lens[b]], **kv1)
        assert ((out[rows, h:h + 1].cpu().double() - want).abs() <= tol).all()
        got = lse[h:h + 1, rows].cpu().double()
        assert ((got - wl).abs() <= 2e-5 * (1 + wl.abs())).all()


@pytest.mark.parametrize("new", [1, 64, 300])
def test_attn_paged_bad_pages_and_lengths_keep_outputs(new):
    c = Cache([600, 600, 600, 600], [new] * 4, 1, 64, 32, torch.float16, False)
    q = torch.randn((4 * new, 2, 64), generator=_gen(1)).half()
    good, _ = _check_attn(c, q, True)
    want, _, tol = oracle.attn(q, c.k, c.v, c.table, c.cu, c.lens)
    for what, seq in (("high", 1), ("low", 2)):
        k, v, table, cu, lens, kw = c.device()
        table[seq, 3] = (1 << 30) if what == "high" else -1
        out = torch.full_like(good, 7.0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tm.tilemix_attn_paged(q.cuda(), k, v, table, cu, lens, new, 600,
                              out=out, status=status)
        assert int(status.item()) == BAD_PAGES
        rows = torch.zeros(4 * new, dtype=torch.bool)
        rows[seq * new:(seq + 1) * new] = True
        assert torch.equal(out[~rows.cuda()], good[~rows.cuda()])
        assert (out[rows.cuda()] == 7).all()
    for lens_bad in ([600, 601, 600, 600], [600, -1, 600, 600],
                     [600, 1 << 30, 600, 600]):
        k, v, table, cu, _, kw = c.device()
        out = torch.full_like(good, 7.0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tm.tilemix_attn_paged(
            q.cuda(), k, v, table, cu,
            torch.tensor(lens_bad, dtype=torch.int32).cuda(), new, 600,
            out=out, status=status)
        assert int(status.item()) == BAD_SEQLENS
        # without the bad sequence the keys split over the blocks elsewhere,
        # so the sums' order may differ; both sides hold the oracle's bound
        near = (out.cpu().double() - want).abs() <= tol
        assert near[:new].all() and near[2 * new:].all()
        assert (out[new:2 * new] == 7).all()


@pytest.mark.parametrize("new", [1, 200])
def test_attn_paged_graph_replays_with_new_lengths(new):
    # one capture serves every step: lengths, table and data are read on the
    # device, max_kv_len is only a bound
    a = Cache([700, 650], [new, new], 2, 128, 16, torch.bfloat16, False, seed=1)
    b = Cache([690, 210], [new, new], 2, 128, 16, torch.bfloat16, False, seed=2)
    q = torch.randn((2 * new, 8, 128), generator=_gen(3)).bfloat16()
    k, v, table, cu, lens, _ = a.device()
    n = max(a.k.shape[0], b.k.shape[0])
    pool = lambda x: torch.cat((x, torch.zeros((n - x.shape[0],) + x.shape[1:],
                                               dtype=x.dtype, device="cuda")))
    k, v = pool(k), pool(v)
    qd = q.cuda()
    out = torch.empty_like(qd)
    lse = torch.empty((8, 2 * new), device="cuda")
    ws = torch.empty(tm.tilemix_attn_paged_workspace_bytes(new, 8, 2, 128),
                     dtype=torch.uint8, device="cuda")
    call = lambda: tm.tilemix_attn_paged(qd, k, v, table, cu, lens, new, 700,
                                         out=out, lse=lse, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    kb, vb, tb, _, lb, _ = b.device()
    w = min(tb.shape[1], table.shape[1])
    k[:kb.shape[0]], v[:vb.shape[0]] = kb, vb
    table[:, :w] = tb[:, :w]
    lens.copy_(lb)
    graph.replay()
    torch.cuda.synchronize()
    want, _ = _check_attn(b, q, True)
    assert torch.equal(out, want)      # same lengths, same order of sums


@pytest.mark.parametrize("new", [1, 150])
def test_attn_paged_two_streams_at_once_and_repeatable(new):
    c = Cache([900, 3000], [new, new], 2, 128, 64, torch.float16, True, seed=4)
    q = torch.randn((2 * new, 16, 128), generator=_gen(5)).half()
    d = c.device()
    want, wl = _check_attn(c, q, True, device=d)
    k, v, table, cu, lens, kw = d
    qd = q.cuda()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(5):
        for s in streams:
            outs.append(tm.tilemix_attn_paged(qd, k, v, table, cu, lens, new,
                                              3000, stream=s, **kw))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_attn_paged_long_cache_offsets_past_31_bits():
    # pages at element offsets above 2^31: 2.2e9 fp16 elements a tensor
    hkv, d, page = 8, 128, 64
    n = (1 << 31) // (page * hkv * d) + 64
    k = torch.empty((n, page, hkv, d), dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    c = Cache([200, 90], [1, 40], hkv, d, page, torch.float16, False, seed=6)
    m = c.k.shape[0]
    k[n - m:], v[n - m:] = c.k.cuda(), c.v.cuda()
    assert (n - m) * page * hkv * d > 1 << 31
    table = torch.where(c.table >= 0, c.table + (n - m), c.table).cuda()
    _, _, _, cu, lens, _ = c.device()
    q = torch.randn((41, 8, d), generator=_gen(7)).half()
    _check_attn(c, q, True, device=(k, v, table, cu, lens, {}))
    # and the append reaches them
    kn = torch.randn((41, hkv, d), generator=_gen(8)).half()
    tm.tilemix_paged_append(kn.cuda(), (kn * 2).cuda(), table, cu, lens, k, v)
    for t, b, p, pid, slot in oracle.places(c.cu, c.lens, table.tolist(), page):
        assert torch.equal(k[pid, slot].cpu(), kn[t])
        assert torch.equal(v[pid, slot].cpu(), kn[t] * 2)


# ---------------------------------------------------------------------------
# appending
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["same", "int8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rot,layout", [(0, "half"), (32, "interleaved"),
                                        (64, "half"), (16, "half")])
@pytest.mark.parametrize("new,lens,hq,hkv,d,page", [
    ([1], [1], 1, 1, 64, 16),
    ([1, 0, 1, 1], [33, 5, 16, 17], 8, 2, 128, 16),
    ([7, 0, 0, 300, 1], [20, 0, 9, 300, 1], 28, 4, 128, 32),
    ([1200, 40], [1201, 99], 3, 1, 64, 64),
    ([5] * 70, [5 + i for i in range(70)], 2, 2, 64, 16),
])
def test_append(new, lens, hq, hkv, d, page, rot, layout, dtype, kv):
    t = TYPES[dtype]
    int8 = kv == "int8"
    c = Cache(lens, new, hkv, d, page, t, int8, seed=len(lens),
              layout=("token", "head", "padded")[len(lens) % 3], poison=False)
    n = c.cu[-1]
    pad = 3
    qkv = torch.randn((n + pad, hq + 2 * hkv, d), generator=_gen(n)).to(t)
    qkv[0, hq:, :] = 0  # a zero row: scale 0, codes 0
    dev = qkv.cuda()
    k, v, table, cu, ln, scales = c.device()
    before = [x.clone() for x in (k, v)]
    freqs = _freqs(rot) if rot else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = torch.full((n + pad, hq, d), 7.0, dtype=t, device="cuda") if rot else None
    got = tm.tilemix_paged_append(
        dev[:, hq:hq + hkv], dev[:, hq + hkv:], table, cu, ln, k, v,
        q=dev[:, :hq] if rot else None, q_out=qo, layout=layout,
        freqs=freqs.cuda() if rot else None, status=status, **scales)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    places = oracle.places(c.cu, c.lens, c.table.tolist(), page)
    pos = torch.tensor([p[2] for p in places], dtype=torch.int32)
    kn, vn = qkv[:n, hq:hq + hkv], qkv[:n, hq + hkv:]
    if rot:
        # the same rotation as the rotary call, bit for bit; that one is
        # checked against the oracle
        rq, rk = tm.tilemix_rope(dev[:n, :hq], dev[:n, hq:hq + hkv], pos.cuda(),
                                 freqs.cuda(), layout=layout)
        assert torch.equal(got[:n], rq) and (got[n:] == 7).all()
        kn = rk.cpu()
    else:
        assert got is None
    ids = torch.tensor([p[3] for p in places])
    slots = torch.tensor([p[4] for p in places])
    for name, rows, pages, old in (("k", kn, k, before[0]),
                                   ("v", vn, v, before[1])):
        want = old.cpu().clone()
        if int8:
            codes, sc = oracle.quantised(rows)
            want[ids, slots] = codes
            ws = (c.ks if name == "k" else c.vs).clone()
            ws[ids, :, slots] = sc
            assert torch.equal(scales[name + "_scale"].cpu(), ws)
        else:
            want[ids, slots] = rows
        assert torch.equal(pages.cpu(), want)


@pytest.mark.parametrize("kv", ["same", "int8"])
def test_append_explicit_positions_and_bad_arguments(kv):
    int8 = kv == "int8"
    c = Cache([40, 40, 40], [3, 3, 3], 2, 64, 16, torch.float16, int8,
              poison=False)
    x = torch.randn((9, 2, 64), generator=_gen(2)).half().cuda()
    pos = torch.tensor([9, 8, 7, 1, 2, 3, 100000, 0, 5], dtype=torch.int32).cuda()
    f = _freqs(64).cuda()
    k, v, table, cu, lens, sc = c.device()
    tm.tilemix_paged_append(x, x, table, cu, lens, k, v, positions=pos, freqs=f,
                            **sc)
    rk, _ = tm.tilemix_rope(x, None, pos, f)
    places = oracle.places(c.cu, c.lens, c.table.tolist(), 16)
    for t, b, p, pid, slot in places:
        row = oracle.quantised(rk[t].cpu())[0] if int8 else rk[t].cpu()
        assert torch.equal(k[pid, slot].cpu(), row)
    # a bad page skips its tokens, a bad length its sequence
    for bad in ("page", "len", "short"):
        k, v, table, cu, lens, sc = c.device()
        k0 = k.clone()
        if bad == "page":
            table[1, 2] = 1 << 20
        else:
            lens[1] = 10000 if bad == "len" else 2
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tm.tilemix_paged_append(x, x, table, cu, lens, k, v, status=status, **sc)
        assert int(status.item()) == (BAD_PAGES if bad == "page" else BAD_SEQLENS)
        want = k0.cpu()
        for t, b, p, pid, slot in places:
            if b != 1:
                row = oracle.quantised(x[t].cpu())[0] if int8 else x[t].cpu()
                want[pid, slot] = row
        assert torch.equal(k.cpu(), want)


# ---------------------------------------------------------------------------
# together: a serving loop
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["same", "int8"])
def test_prefill_chunks_and_decode_steps(kv):
    """Two prompts enter the cache in chunks, then decode together; every
    token's output equals causal attention over everything appended."""
    int8 = kv == "int8"
    hq, hkv, d, page = 8, 2, 64, 16
    t = torch.float16
    g = _gen(12)
    n = [75, 40]
    steps = [([40, 1], [40, 1]), ([30, 30], [70, 31]), ([4, 8], [74, 39]),
             ([1, 1], [75, 40])]
    xs = [torch.randn((m, hq + 2 * hkv, d), generator=g).to(t) for m in n]
    freqs, att = tm.tilemix_rope_frequencies(
        d, 10000.0, scaling="wavelength", factor=8.0, low_freq_factor=1.0,
        high_freq_factor=4.0, original_max_position=64, device="cuda")
    assert att == 1.0
    table = torch.tensor([[3, 0, 5, 9, 1], [7, 2, 8, -1, -1]],
                         dtype=torch.int32).cuda()
    kp = torch.zeros((10, page, hkv, d), dtype=torch.int8 if int8 else t,
                     device="cuda")
    vp = torch.zeros_like(kp)
    sc = {}
    if int8:
        sc = dict(k_scale=torch.zeros((10, hkv, page), device="cuda"),
                  v_scale=torch.zeros((10, hkv, page), device="cuda"))
    outs = [[], []]
    rot = [[], []]
    at = [0, 0]
    for new, lens in steps:
        x = torch.cat([xs[b][at[b]:at[b] + new[b]] for b in range(2)]).cuda()
        cu = torch.tensor([0, new[0], sum(new)], dtype=torch.int32).cuda()
        ln = torch.tensor(lens, dtype=torch.int32).cuda()
        q = tm.tilemix_paged_append(x[:, hq:hq + hkv], x[:, hq + hkv:], table,
                                    cu, ln, kp, vp, q=x[:, :hq], freqs=freqs,
                                    layout="interleaved", **sc)
        o = tm.tilemix_attn_paged(q, kp, vp, table, cu, ln, max(new), max(lens),
                                  **sc)
        for b, s in ((0, slice(0, new[0])), (1, slice(new[0], sum(new)))):
            outs[b].append(o[s].cpu())
            rot[b].append(q[s].cpu())
            at[b] += new[b]
            assert at[b] == lens[b]
    for b in range(2):
        want, _, tol = oracle.attn(
            torch.cat(rot[b]), kp.cpu(), vp.cpu(), [table[b].tolist()],
            [0, n[b]], [n[b]], **{x: y.cpu() for x, y in sc.items()})
        got = torch.cat(outs[b]).double()
        assert ((got - want).abs() <= tol).all()
