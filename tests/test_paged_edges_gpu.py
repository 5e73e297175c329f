"""The serving operators on the GPU where they can go wrong at the edges: side streams, queries
and caches of wide range, bad pages, NaN and huge values, lengths without tokens.  Definitions
and tolerances are those of ``test_paged_gpu``."""
import math

import pytest
import torch

from tests import paged_reference as ref
from tests.test_paged_gpu import Pool, attn, bounds, check_attention, ints, normal, ok  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ streams
BUSY = 50_000_000        # cycles for which the current stream is kept busy


@pytest.mark.parametrize("e4m3", [False, True])
def test_reading_on_a_side_stream_keeps_its_rows(attn, e4m3):  # noqa: F811
    """The zeros behind a sequence come before the rows, also while the current stream is busy."""
    lens, N = [150, 0, 33], 160
    pool = Pool(3, 2, 32, 64, lens, e4m3, seed=5)
    where, scales = pool.cuda()
    kv_len = ints(lens).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    k, v = attn.attn_cache_read(*where, kv_len, **scales, N=N, stream=side)
    torch.cuda.synchronize()
    ok(attn)
    for b, L in enumerate(lens):
        for got, n in ((k, "k"), (v, "v")):
            assert torch.equal(got[b, :, :L].cpu().double(), ref.gathered(pool.value[n], pool.table[b], L))
            assert bool((got[b, :, L:] == 0).all())


def test_outputs_on_a_side_stream_are_not_memory_that_others_still_write(attn):  # noqa: F811
    """Freed blocks of the outputs' sizes with writes still queued on the current stream."""
    T, Hq, Hkv, d, L = 40, 4, 2, 64, 300
    pool = Pool(1, Hkv, 32, d, [L], False, seed=6)
    (kc, vc, table), _ = pool.cuda()
    q, k, v = (normal((T, H, d), 60 + H + i).cuda() for i, H in enumerate((Hq, Hkv, Hkv)))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    f = attn.rope_inv_freq(d)[0]
    cu, kv_len = bounds([T]).cuda(), ints([L]).cuda()
    calls = [lambda **kw: attn.attn_rope(q, k, positions=pos, inv_freq=f, **kw),
             lambda **kw: (attn.attn_cache_write(k, v, kc, vc, table, cu, kv_len, inv_freq=f, q=q, **kw),),
             lambda **kw: attn.attn_paged(q, kc, vc, table, cu, kv_len, **kw)]
    side = torch.cuda.Stream()
    for call in calls:
        call()                                  # (the write leaves the same cache each time)
        want = [x.clone() for x in call()]
        torch.cuda.synchronize()
        blocks = [torch.empty_like(x) for x in want for _ in range(2)]
        torch.cuda._sleep(BUSY)
        for b in blocks:
            b.fill_(7.0)
        del blocks, b
        got = call(stream=side)
        torch.cuda.synchronize()
        ok(attn)
        assert all(torch.equal(g, w) for g, w in zip(got, want))
