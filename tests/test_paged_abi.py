"""Rotary and paged-cache calls without a GPU: the Python structs mirror the
C layout, host checks refuse bad calls before any launch, the binding refuses
wrong tensors, the frequency helper agrees with its formulas, and the oracle
is pinned to dense textbook forms."""
import ctypes as C
import math
import os
import subprocess
import tempfile

import pytest

tm = pytest.importorskip("prefill_blockwise_int8_b200")
torch = pytest.importorskip("torch")

from oracle import paged as oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, NO_DEVICE = 0, 1, 2, 6
FAKE = 0x10000  # 16-byte aligned, never dereferenced on the host
DEVICE_VISIBLE = torch.cuda.is_available()


def accepted(fn, *args):
    # with a device a call that passes the checks would launch on fake pointers
    return DEVICE_VISIBLE or fn(*args) == NO_DEVICE


@pytest.mark.parametrize("struct,name", [
    (tm.RopeParams, "tilemix_rope_params"),
    (tm.AppendParams, "tilemix_append_params"),
    (tm.AttnPagedParams, "tilemix_attn_paged_params")])
def test_struct_layout_matches_c(struct, name):
    fields = [f for f, _ in struct._fields_]
    prog = ["#include <stdio.h>", "#include <stddef.h>", '#include "tilemix.h"',
            "int main(void) {", f'printf("size %zu\\n", sizeof({name}));']
    prog += [f'printf("{f} %zu\\n", offsetof({name}, {f}));' for f in fields]
    prog.append("return 0; }")
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "layout.c"), os.path.join(d, "layout")
        open(src, "w").write("\n".join(prog))
        subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I",
                        os.path.join(ROOT, "include"), src, "-o", exe],
                       check=True)
        out = subprocess.run([exe], capture_output=True, text=True,
                             check=True).stdout
    got = dict(line.split() for line in out.strip().splitlines())
    assert int(got["size"]) == C.sizeof(struct)
    for f in fields:
        assert int(got[f]) == getattr(struct, f).offset, f


def test_status_string():
    assert tm.tilemix_status_string(7) == "invalid page table entry"


def make(struct, good, over):
    p = struct()
    p.struct_size = C.sizeof(struct)
    for k, v in dict(good, **over).items():
        setattr(p, k, v)
    return p


ROPE = dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, q_stride_t=1024,
            q_stride_h=128, k_stride_t=256, k_stride_h=128,
            q_out_stride_t=1024, q_out_stride_h=128, k_out_stride_t=256,
            k_out_stride_h=128, positions=FAKE, freqs=FAKE, attn_factor=1.0,
            total_tokens=5, hq=8, hkv=2, head_dim=128, rot_dim=128)


def rope(**over):
    return tm.lib.tilemix_rope(C.byref(make(tm.RopeParams, ROPE, over)), None)


def test_rope_accepts():
    assert accepted(rope)
    assert accepted(lambda: rope(k=0, k_out=0, hkv=0))
    assert accepted(lambda: rope(head_dim=80, rot_dim=16))
    assert rope(total_tokens=0, q=0, freqs=0) == OK
    assert tm.lib.tilemix_rope(None, None) == INVALID


@pytest.mark.parametrize("over,expect", [
    (dict(struct_size=8), INVALID), (dict(dtype=2), INVALID),
    (dict(layout=2), INVALID), (dict(inverse=2), INVALID),
    (dict(q=0), INVALID), (dict(q_out=0), INVALID), (dict(k_out=0), INVALID),
    (dict(positions=0), INVALID), (dict(freqs=0), INVALID),
    (dict(freqs=FAKE + 4), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(k_out=FAKE + 2), INVALID), (dict(q_stride_h=132), INVALID),
    (dict(q_stride_t=-8), INVALID), (dict(k_out_stride_t=4), INVALID),
    (dict(q_out_stride_t=0), INVALID), (dict(q_out_stride_h=64), INVALID),
    (dict(k_out_stride_h=0), INVALID),
    (dict(total_tokens=-1), INVALID), (dict(hq=0), INVALID),
    (dict(hkv=0), INVALID), (dict(hq=65535), INVALID),
    (dict(head_dim=72), UNSUPPORTED), (dict(head_dim=272), UNSUPPORTED),
    (dict(head_dim=0), UNSUPPORTED), (dict(rot_dim=24), UNSUPPORTED),
    (dict(rot_dim=144), UNSUPPORTED), (dict(rot_dim=0), UNSUPPORTED),
    (dict(attn_factor=float("nan")), INVALID),
    (dict(attn_factor=float("inf")), INVALID),
    (dict(attn_factor=-1.0), INVALID)])
def test_rope_refuses(over, expect):
    assert rope(**over) == expect
    assert tm.tilemix_last_error()


CACHE = dict(k_pages=FAKE, v_pages=FAKE, page_stride=16 * 256, token_stride=256,
             head_stride=128, page_table=FAKE, table_stride=10, cu_seqlens=FAKE,
             kv_lens=FAKE, batch=3, total_tokens=5, hkv=2, head_dim=128,
             num_pages=30, page_size=16, max_pages=10)
APPEND = dict(CACHE, k=FAKE, v=FAKE, k_stride_t=256, k_stride_h=128,
              v_stride_t=256, v_stride_h=128)
ATTN = dict(CACHE, causal=1, q=FAKE, q_stride_t=1024, q_stride_h=128,
            max_q_len=3, max_kv_len=160, hq=8, out=FAKE, workspace=FAKE,
            workspace_bytes=1 << 40)


def append(**over):
    return tm.lib.tilemix_paged_append(
        C.byref(make(tm.AppendParams, APPEND, over)), None)


def attn(**over):
    return tm.lib.tilemix_attn_paged(
        C.byref(make(tm.AttnPagedParams, ATTN, over)), None)


def test_cache_calls_accept():
    assert accepted(append) and accepted(attn)
    assert accepted(lambda: append(q=FAKE, q_out=FAKE, hq=8, freqs=FAKE,
                                   rot_dim=64, q_stride_t=1024, q_stride_h=128,
                                   q_out_stride_t=1024, q_out_stride_h=128))
    for call in (append, attn):
        assert accepted(lambda: call(kv_format=1, k_scale=FAKE, v_scale=FAKE))
        assert accepted(lambda: call(page_size=256, head_dim=64))
        assert call(batch=0) == OK and call(total_tokens=0) == OK
    assert attn(max_q_len=0) == OK
    assert tm.lib.tilemix_paged_append(None, None) == INVALID
    assert tm.lib.tilemix_attn_paged(None, None) == INVALID


@pytest.mark.parametrize("over,expect", [
    (dict(struct_size=8), INVALID), (dict(dtype=2), INVALID),
    (dict(kv_format=2), INVALID), (dict(kv_format=1), INVALID),
    (dict(kv_format=1, k_scale=FAKE, v_scale=FAKE + 4), INVALID),
    (dict(kv_format=1, k_scale=FAKE, v_scale=FAKE, token_stride=264), INVALID),
    (dict(k_pages=0), INVALID), (dict(v_pages=FAKE + 8), INVALID),
    (dict(page_table=0), INVALID), (dict(cu_seqlens=0), INVALID),
    (dict(kv_lens=0), INVALID), (dict(kv_lens=FAKE + 2), INVALID),
    (dict(status=FAKE + 2), INVALID),
    (dict(batch=-1), INVALID), (dict(total_tokens=-1), INVALID),
    (dict(hkv=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(table_stride=9), INVALID),
    (dict(page_stride=100), INVALID), (dict(token_stride=64), INVALID),
    (dict(token_stride=132), INVALID), (dict(head_stride=64), INVALID),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
    (dict(page_size=512), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
    (dict(head_dim=256), UNSUPPORTED), (dict(max_pages=1 << 27), UNSUPPORTED)])
def test_cache_calls_refuse(over, expect):
    assert append(**over) == expect
    assert tm.tilemix_last_error()
    assert attn(**over) == expect
    assert tm.tilemix_last_error()


@pytest.mark.parametrize("over,expect", [
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(layout=3), INVALID),
    (dict(q=FAKE, hq=8), INVALID), (dict(v_stride_t=12), INVALID),
    (dict(freqs=FAKE, rot_dim=144), UNSUPPORTED),
    (dict(freqs=FAKE, rot_dim=8), UNSUPPORTED),
    (dict(freqs=FAKE + 4, rot_dim=64), INVALID),
    (dict(positions=FAKE + 1), INVALID), (dict(attn_factor=-1.0), INVALID)])
def test_append_refuses(over, expect):
    assert append(**over) == expect


@pytest.mark.parametrize("over,expect", [
    (dict(q=0), INVALID), (dict(out=0), INVALID), (dict(out=FAKE + 8), INVALID),
    (dict(lse=FAKE + 2), INVALID), (dict(hq=7), INVALID), (dict(hq=0), INVALID),
    (dict(hq=258), UNSUPPORTED), (dict(causal=2), INVALID),
    (dict(max_q_len=-1), INVALID), (dict(max_kv_len=-1), INVALID),
    (dict(max_q_len=1 << 29), UNSUPPORTED),
    (dict(softmax_scale=float("nan")), INVALID),
    (dict(workspace=0), INVALID), (dict(workspace=FAKE + 8), INVALID),
    (dict(workspace_bytes=100), INVALID), (dict(q_stride_t=1020), INVALID)])
def test_attn_refuses(over, expect):
    assert attn(**over) == expect


def test_workspace_bytes():
    ws = tm.tilemix_attn_paged_workspace_bytes
    assert 0 < ws(1, 32, 8, 64) < ws(1, 32, 8, 128) < 64 << 20
    # it grows with max_q_len at most, so one for the longest call serves all
    sizes = [ws(n, 28, 4, 128) for n in (0, 1, 2, 3, 4, 5, 40, 5000)]
    assert sizes == sorted(sizes)
    for bad in ((-1, 32, 8, 128), (1, 0, 8, 128), (1, 32, 0, 128),
                (1, 30, 8, 128), (1, 32, 8, 96), (1, 129, 1, 128)):
        assert ws(*bad) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 2, 64), dtype=torch.float16)
    i = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(32, dtype=torch.float64)
    pages = torch.zeros((3, 16, 2, 64), dtype=torch.float16)
    for call in (lambda: tm.tilemix_rope(x, x, i, f),
                 lambda: tm.tilemix_paged_append(x, x, i[None], i, i, pages, pages),
                 lambda: tm.tilemix_attn_paged(x, pages, pages, i[None], i, i, 1, 1)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


# ---------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------

def _f(**kw):
    return tm.tilemix_rope_frequencies(64, 10000.0, **kw)


def test_frequencies():
    base, att = _f()
    want = torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)],
                        dtype=torch.float64)
    assert att == 1.0 and base.dtype == torch.float64
    assert torch.allclose(base, want, rtol=1e-14, atol=0)
    lin, _ = _f(scaling="linear", factor=4.0)
    assert torch.allclose(lin, want / 4, rtol=1e-14, atol=0)
    ntk, _ = _f(scaling="ntk", factor=4.0)
    # the longest wavelength grows by the factor, the shortest stays
    assert ntk[0] == 1.0
    assert abs(float(ntk[31] / want[31]) - 0.25) < 1e-12
    wl, _ = _f(scaling="wavelength", factor=8.0, low_freq_factor=1.0,
               high_freq_factor=4.0, original_max_position=8192)
    wave = 2 * math.pi / want
    assert torch.allclose(wl[wave < 2048], want[wave < 2048], rtol=1e-14)
    assert torch.allclose(wl[wave > 8192], want[wave > 8192] / 8, rtol=1e-14)
    assert ((wl <= want) & (wl >= want / 8 * (1 - 1e-12))).all()
    mid = (wave >= 2048) & (wave <= 8192)
    t = (8192 / wave[mid] - 1) / 3
    assert mid.any() and torch.allclose(
        wl[mid], (1 - t) * want[mid] / 8 + t * want[mid], rtol=1e-12)
    yarn, att = _f(scaling="yarn", factor=16.0, low_freq_factor=1.0,
                   high_freq_factor=32.0, original_max_position=4096)
    assert abs(att - (0.1 * math.log(16.0) + 1)) < 1e-6
    dim = lambda n: 64 * math.log(4096 / (n * 2 * math.pi)) / (2 * math.log(1e4))
    lo, hi = max(math.floor(dim(32)), 0), min(math.ceil(dim(1)), 63)
    t = ((torch.arange(32) - lo) / (hi - lo)).clamp(0, 1).double()
    assert torch.allclose(yarn, t * want / 16 + (1 - t) * want, rtol=1e-12)


@pytest.mark.parametrize("kw", [
    dict(scaling=5), dict(scaling=-1), dict(scaling="linear", factor=0.0),
    dict(scaling="linear", factor=float("inf")),
    dict(scaling="yarn", factor=2.0, original_max_position=0),
    dict(scaling="wavelength", factor=2.0, original_max_position=8,
         low_freq_factor=4.0, high_freq_factor=4.0),
    dict(scaling="wavelength", factor=2.0, original_max_position=8,
         low_freq_factor=0.0)])
def test_frequencies_refuse(kw):
    with pytest.raises(tm.TilemixError):
        _f(**kw)


@pytest.mark.parametrize("args", [(0, 10000.0), (7, 10000.0), (-2, 10000.0),
                                  (64, 1.0), (64, float("nan")),
                                  (64, float("inf"))])
def test_frequencies_refuse_sizes(args):
    with pytest.raises(tm.TilemixError):
        tm.tilemix_rope_frequencies(*args)


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------

def test_oracle_rope_is_a_rotation():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((3, 2, 8), generator=g, dtype=torch.float64)
    f = torch.tensor([1.0, 0.5], dtype=torch.float64)
    pos = torch.tensor([0, 1, 9], dtype=torch.int32)
    for layout in ("half", "interleaved"):
        y = oracle.rope(x, pos, f, layout)
        assert torch.equal(y[0], x[0]) and torch.equal(y[..., 4:], x[..., 4:])
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1))
        assert torch.allclose(oracle.rope(y, pos, f, layout, inverse=True), x)
        # scores depend on the distance of the positions only
        a = oracle.rope(x, pos + 5, f, layout) @ oracle.rope(x, pos, f, layout)[..., None].squeeze(-1).transpose(1, 2)
        b = oracle.rope(x, pos + 105, f, layout) @ oracle.rope(x, pos + 100, f, layout)[..., None].squeeze(-1).transpose(1, 2)
        assert torch.allclose(a, b)
    y = oracle.rope(x[1:2], pos[1:2], f, "interleaved")
    assert torch.allclose(y[0, 0, 0], x[1, 0, 0] * math.cos(1) - x[1, 0, 1] * math.sin(1))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("int8", [True, False])
def test_oracle_attention_is_dense_attention(causal, int8):
    g = torch.Generator().manual_seed(1)
    n, m, page, hq, hkv, d = 37, 9, 16, 4, 2, 8
    order = [4, 0, 2]
    k, v = (torch.randn((5, page, hkv, d), generator=g) for _ in range(2))
    kw = {}
    if int8:
        (k, ks), (v, vs) = oracle.quantised(k), oracle.quantised(v)
        kw = dict(k_scale=ks.transpose(1, 2), v_scale=vs.transpose(1, 2))
    q = torch.randn((m, hq, d), generator=g)
    out, lse, tol = oracle.attn(q, k, v, [order + [-1]], [0, m], [n],
                                causal=causal, **kw)
    dense = lambda x, s: ((x.double() * s[..., None].double() if int8 else
                           x.double())[order].flatten(0, 1)[:n]
                          .repeat_interleave(hq // hkv, 1))
    kd, vd = dense(k, ks if int8 else 0), dense(v, vs if int8 else 0)
    s = torch.einsum("ihd,jhd->hij", q.double(), kd) / math.sqrt(d)
    if causal:
        i = torch.arange(m)[:, None] + n - m
        s = s.masked_fill(torch.arange(n)[None] > i, -math.inf)
    want = torch.einsum("hij,jhd->ihd", s.softmax(-1), vd)
    assert torch.allclose(out, want) and torch.allclose(lse, s.logsumexp(-1))
    assert (tol > 0).all()


def test_attn_flags():
    assert accepted(lambda: attn(flags=tm.FLAG_TEST_EXPIRE_WAIT))
    for bad in (1, 2, 8, 1 << 31):
        assert attn(flags=bad) == INVALID and "flags" in tm.tilemix_last_error()
    # the field fills what was padding: no other one moved
    assert C.sizeof(tm.AttnPagedParams) == 216


@pytest.mark.parametrize("over", [
    dict(q_out_stride_t=128, q_out_stride_h=128),   # row t, h = row t + h
    dict(q_out_stride_t=256, q_out_stride_h=128),
    dict(k_out_stride_t=128, k_out_stride_h=256),
    dict(q_out_stride_t=128, q_out_stride_h=512),
    dict(q_out_stride_t=1016), dict(k_out_stride_t=248)])
def test_rope_refuses_outputs_that_overlap(over):
    assert rope(**over) == INVALID and "overlap" in tm.tilemix_last_error()


def test_outputs_may_lie_either_way():
    assert accepted(lambda: rope(q_out_stride_t=128, q_out_stride_h=5 * 128))
    assert accepted(lambda: rope(q_out_stride_t=1 << 40, q_out_stride_h=136))
    assert accepted(lambda: rope(total_tokens=1, q_out_stride_t=0))
    assert accepted(lambda: rope(hq=1, q_out_stride_h=0, q_out_stride_t=128))
    # pages: token-major (above), head-major, heads outermost, one page, K and
    # V interleaved by page, slot or head
    for sp, st, sh, over in [
            (16 * 256, 128, 16 * 128, {}), (16 * 128, 128, 30 * 16 * 128, {}),
            (0, 256, 128, dict(num_pages=1)), (16 * 256, 256, 0, dict(hkv=1)),
            (2 * 16 * 256, 256, 128, {}), (2 * 16 * 256, 512, 128, {}),
            (2 * 16 * 256, 512, 256, {})]:
        assert accepted(lambda: append(page_stride=sp, token_stride=st,
                                       head_stride=sh, **over))


@pytest.mark.parametrize("sp,st,sh", [
    (16 * 256, 128, 128), (16 * 256, 256, 256), (16 * 256, 248, 128),
    (16 * 256, 136, 128), (16 * 256, 128, 15 * 128), (16 * 256, 128, 256)])
def test_append_refuses_pages_that_overlap(sp, st, sh):
    assert append(page_stride=sp, token_stride=st, head_stride=sh) == INVALID
    assert "overlap" in tm.tilemix_last_error()
    # reading them is well defined
    assert accepted(lambda: attn(page_stride=sp, token_stride=st, head_stride=sh))


def test_positions_stay_inside_32_bits():
    # unit ends and the keys a copy looks ahead are int32 too
    most = ((1 << 31) - 1024) // 16
    for call in (append, attn):
        assert accepted(lambda: call(max_pages=most, table_stride=most))
        for n in (most + 1, (1 << 27) - 1):
            assert call(max_pages=n, table_stride=n) == UNSUPPORTED


def test_sizes_beyond_32_bits():
    ws = tm.tilemix_attn_paged_workspace_bytes
    for n in ((1 << 32) + 1, 1 << 31, (1 << 30) // 4 + 1):
        assert ws(n, 8, 2, 128) == 0
    assert ws((1 << 30) // 4, 8, 2, 128) > 0
    assert ws(1, (1 << 32) + 8, 2, 128) == 0
    q, pages = torch.empty((1, 8, 128)), torch.empty((1, 16, 2, 128))
    with pytest.raises(ValueError, match="CUDA tensor"):
        tm.tilemix_attn_paged(q, pages, pages, None, None, None, 1 << 31, 1)
