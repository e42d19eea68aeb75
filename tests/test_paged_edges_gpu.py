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
