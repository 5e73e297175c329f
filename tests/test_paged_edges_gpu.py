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


# ------------------------------------------------------------------ queries of wide range
FEW = [   # Hq / Hkv, tokens per sequence: every build of the kernel for few rows, then one of the 128-row kernel
    (1, 1), (4, 1), (2, 3), (8, 1), (3, 5), (16, 1)]


@pytest.mark.parametrize("wide", [0, 10, 13, 17, 27])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", FEW)
def test_small_channels_of_a_wide_query_keep_their_bits_over_e4m3(attn, G, n, d, wide):  # noqa: F811
    """One channel of Q 2^wide times the others, where K is small (codes of 0 to 3 units of 2^-9; all
    zero at 2^27): the others decide the scores and must not lose bits to the large one."""
    B, Hkv, page, lens = 2, 2, 32, [300, 129]
    pool = Pool(B, Hkv, page, d, lens, True, seed=wide + d)
    g = torch.Generator().manual_seed(9)
    small = torch.randint(0, 4 if wide < 20 else 1, pool.store["k"].shape[:3], generator=g).to(torch.uint8)
    own = pool.store["k"][..., 5] != 0x7f
    pool.store["k"][..., 5] = torch.where(own, small, pool.store["k"][..., 5])
    pool.value["k"] = ref.widened(pool.store["k"], pool.store["ks"])
    q = normal((B * n, G * Hkv, d), 3 + G)
    q[..., 5] = (q[..., 5].float().abs() + 0.5).mul(2.0 ** wide).to(torch.bfloat16)
    where, scales = pool.cuda()
    got = attn.attn_paged(q.cuda(), *where, bounds([n] * B).cuda(), ints(lens).cuda(), **scales)
    ok(attn)
    check_attention(got, ref.attend(q, pool.value["k"], pool.value["v"], pool.table, bounds([n] * B), lens, d ** -0.5))


@pytest.mark.parametrize("d", [64, 128])
def test_an_answer_over_e4m3_does_not_depend_on_the_rows_of_the_call(attn, d):  # noqa: F811
    """The same wide query alone (few rows) and beside 200 other tokens (the 128-row kernel).  Both round
    P and O once: they differ by two roundings of each at most."""
    Hq, Hkv, page, L = 4, 1, 64, 700
    pool = Pool(2, Hkv, page, d, [L, 200], True, seed=d)
    pool.store["k"][..., 9] = torch.where(pool.store["k"][..., 9] != 0x7f, 1, pool.store["k"][..., 9])
    pool.value["k"] = ref.widened(pool.store["k"], pool.store["ks"])
    q = normal((201, Hq, d), 4)
    q[..., 9] = (q[..., 9].float() * 2.0 ** 15).to(torch.bfloat16)
    (kc, vc, table), scales = pool.cuda()
    one = attn.attn_paged(q[:1].cuda(), kc, vc, table[:1].contiguous(), bounds([1]).cuda(), ints([L]).cuda(), **scales)
    many = attn.attn_paged(q.cuda(), kc, vc, table, bounds([1, 200]).cuda(), ints([L, 200]).cuda(), **scales)
    ok(attn)
    wo, wl, wabs = ref.attend(q[:1], pool.value["k"], pool.value["v"], pool.table, bounds([1]), [L], d ** -0.5)
    check_attention(one, (wo, wl, wabs))
    assert float((one[1] - many[1][:1]).abs().max()) <= 1e-3
    u = 2.0 ** -8
    diff = (one[0].cpu().double() - many[0][:1].cpu().double()).abs()
    assert bool((diff <= 2 * ((u + 2e-4) * wabs + u * wo.abs()) + 1e-6).all())


@pytest.mark.parametrize("power,byte", [(119, 3), (-110, 230)])
@pytest.mark.parametrize("G,n", FEW)
def test_huge_and_tiny_scales_cancel_over_e4m3(attn, G, n, power, byte):  # noqa: F811
    """Queries of 2^power against keys of about 2^-power: scores of a few units, though the sum of
    codes and one of the two scales alone can leave fp32's range."""
    B, Hkv, d, page, lens = 2, 2, 128, 16, [300, 129]
    pool = Pool(B, Hkv, page, d, lens, True, seed=G + n)
    codes = pool.store["k"]
    codes[(codes & 0x78) <= 0x68] += 16                        # four times the value; NaN stays
    pool.store["ks"] = pool.store["ks"] - 119 + byte           # byte .. byte + 4
    pool.value["k"] = ref.widened(codes, pool.store["ks"])
    q = (normal((B * n, G * Hkv, d), 3 + G, torch.float32) * 2.0 ** power).to(torch.bfloat16)
    where, scales = pool.cuda()
    scale = d ** -0.5 / 32                                     # sums of sizes up to 13: the tolerance holds
    got = attn.attn_paged(q.cuda(), *where, bounds([n] * B).cuda(), ints(lens).cuda(), **scales, scale=scale)
    ok(attn)
    want = ref.attend(q, pool.value["k"], pool.value["v"], pool.table, bounds([n] * B), lens, scale)
    finite = want[1][~torch.isinf(want[1])]
    assert bool((finite.abs() < 30).all())                     # the case is one of ordinary scores
    check_attention(got, want)


# ------------------------------------------------------------------ pages that are not followed
@pytest.mark.parametrize("Hq", [1, 8, 16, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_bad_pages_over_e4m3_count_as_zeros_whatever_was_loaded_before(attn, d, Hq):  # noqa: F811
    """3000 one-page sequences, some 20 to an SM: eight of good pages under the scale byte 255
    (infinity), then eight whose table entry is no page.  The latter see 16 keys of zeros."""
    B, page = 3000, 16
    kc, vc = (torch.ones(2, 1, page, d, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full((2, 1, page), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    b = torch.arange(B)
    bad = (b // 8) % 2 == 1
    table = torch.where(bad, torch.where(b % 2 == 0, -1, 2), b % 2).to(torch.int32).reshape(B, 1).cuda()
    q = normal((B, Hq, d), 3).cuda()
    o, lse = attn.attn_paged(q, kc, vc, table, torch.arange(B + 1, dtype=torch.int32, device="cuda"),
                             torch.full((B,), page, dtype=torch.int32, device="cuda"), k_scale=ks, v_scale=vs)
    assert attn.attn_get_device_status() == -10
    assert bool((o.cpu()[bad] == 0).all())
    assert float((lse.cpu()[bad] - math.log(page)).abs().max()) <= 1e-5
    ok(attn)


# ------------------------------------------------------------------ values that are not finite, or huge
FORMS = [(4, 1), (2, 20), (2, 100)]         # Hq / Hkv, tokens: the kernels for few rows, 128 rows, two tiles of 128


@pytest.mark.parametrize("e4m3,bad", [(False, math.nan), (False, math.inf), (True, math.nan)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", FORMS)
def test_a_key_that_is_not_finite_reaches_the_rows_that_see_it_and_no_others(attn, G, n, d, e4m3, bad):  # noqa: F811
    """16 sequences with such a value in one channel of the key at one of 16 successive positions, so at
    every column of a softmax thread's loop.  Rows that see it are NaN, or for a score of -inf
    free of it, as the definition says; the others are untouched."""
    B, Hkv, page, L = 16, 1, 32, 300
    pool = Pool(B, Hkv, page, d, [L] * B, e4m3, seed=d + n)
    for b in range(B):
        p = 230 + b
        at = (int(pool.table[b, p // page]), 0, p % page, 11)
        pool.store["k"][at] = 0x7f if e4m3 else bad
    pool.value["k"] = ref.widened(pool.store["k"], pool.store["ks"]) if e4m3 else pool.store["k"].double()
    q = normal((B * n, G, d), 5)
    where, scales = pool.cuda()
    o, lse = (x.cpu().double() for x in attn.attn_paged(q.cuda(), *where, bounds([n] * B).cuda(), ints([L] * B).cuda(), **scales))
    ok(attn)
    wo, wl, wabs = ref.attend(q, pool.value["k"], pool.value["v"], pool.table, bounds([n] * B), [L] * B, d ** -0.5)
    seen = wo.isnan().any(-1)                              # [T, Hq]
    assert bool(seen.any()) and torch.equal(o.isnan().all(-1), seen) and torch.equal(o.isnan().any(-1), seen)
    assert bool((~lse[seen].isfinite()).all())
    check_attention((o[~seen], lse[~seen]), (wo[~seen], wl[~seen], wabs[~seen]))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", FORMS)
def test_huge_values_at_masked_positions_do_not_leak(attn, G, n, d, e4m3):  # noqa: F811
    """V of the type's largest magnitude at every position that a row does not see (later new tokens,
    positions before the window) must add nothing: the rows that see none of it agree with the
    definition to their own tolerance."""
    B, Hkv, page, L, window = 3, 1, 32, 400, 60
    pool = Pool(B, Hkv, page, d, [L] * B, e4m3, seed=d + n)
    first = L - n
    far = first - window                                   # the first row's window begins here
    huge = list(range(far - 30, far)) + list(range(first + 1, L))     # the first row sees none of them
    for b in range(B):
        for p in huge:
            at = (int(pool.table[b, p // page]), slice(None), p % page)
            if e4m3:
                pool.store["v"][at] = 0x7e                 # 448 under the largest scale the write makes
                pool.store["vs"][at] = 247 - 1
            else:
                pool.store["v"][at] = torch.finfo(torch.bfloat16).max * (-1) ** p
    pool.value["v"] = ref.widened(pool.store["v"], pool.store["vs"]) if e4m3 else pool.store["v"].double()
    q = normal((B * n, G, d), 5)
    where, scales = pool.cuda()
    o, lse = (x.cpu() for x in attn.attn_paged(q.cuda(), *where, bounds([n] * B).cuda(), ints([L] * B).cuda(), **scales,
                                               window_left=window))
    ok(attn)
    want = ref.attend(q, pool.value["k"], pool.value["v"], pool.table, bounds([n] * B), [L] * B, d ** -0.5, True, window)
    rows = torch.arange(0, B * n, n)                       # of each sequence the first
    check_attention((o[rows], lse[rows]), tuple(x[rows] for x in want))
    assert float(want[0][rows].abs().max()) < 10


# ------------------------------------------------------------------ lengths
@pytest.mark.parametrize("length", [-1, -5, -(1 << 30), -(1 << 31)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_a_negative_length_counts_as_zero(attn, length, e4m3):  # noqa: F811
    """Nothing is written, read or attended to for that sequence and nothing is reported; the other one's
    results are those of the call alone."""
    Hq, Hkv, d, page, L, n = 4, 2, 64, 16, 40, 3
    pool = Pool(1, Hkv, page, d, [L], e4m3, seed=3)
    (kc, vc, table), scales = pool.cuda()
    rows = normal((2 * n, Hq + 2 * Hkv, d), 4).cuda()
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    kc2, vc2 = kc.clone(), vc.clone()
    sc2 = {m: x.clone() for m, x in scales.items()}
    alone = (bounds([n]).cuda(), ints([L]).cuda())
    both = (bounds([n, n]).cuda(), ints([L, length]).cuda())
    t2 = table.repeat(2, 1).contiguous()
    attn.attn_cache_write(k[:n], v[:n], kc, vc, table, *alone, **scales)
    attn.attn_cache_write(k, v, kc2, vc2, t2, *both, **sc2)
    ok(attn)
    for a, b in [(kc, kc2), (vc, vc2)] + [(scales[m], sc2[m]) for m in scales]:
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    want = attn.attn_paged(q[:n], kc, vc, table, *alone, **scales)
    got = attn.attn_paged(q, kc, vc, t2, *both, **scales)
    kr, vr = attn.attn_cache_read(kc, vc, t2, both[1], N=L, **scales)
    ok(attn)
    assert all(torch.equal(g[:n], w) for g, w in zip(got, want))
    assert bool((got[0][n:] == 0).all()) and bool(torch.isinf(got[1][n:]).all())
    assert bool((kr[1] == 0).all()) and bool((vr[1] == 0).all())


@pytest.mark.parametrize("T", [1, 40, 300])
def test_a_slot_without_tokens_is_not_reported_for_its_length(attn, T):  # noqa: F811
    """Slots that wait (no new token) may hold any length: no row sees a position behind their table."""
    Hq, Hkv, d, page, L = 4, 2, 64, 16, 330
    pool = Pool(1, Hkv, page, d, [L], False, seed=3)
    (kc, vc, table), _ = pool.cuda()
    q = normal((T, Hq, d), 4)
    got = attn.attn_paged(q.cuda(), kc, vc, table.repeat(3, 1).contiguous(), bounds([0, T, 0]).cuda(),
                          ints([1 << 29, L, page * table.shape[1] + 1]).cuda())
    ok(attn)
    check_attention(got, ref.attend(q, pool.value["k"], pool.value["v"], pool.table, bounds([T]), [L], d ** -0.5))


# ------------------------------------------------------------------ running maxima
@pytest.mark.parametrize("order", ["rising", "falling", "one"])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", FEW + [(2, 20), (2, 100)])
def test_maxima_that_move_from_tile_to_tile(attn, G, n, d, e4m3, order):  # noqa: F811
    """Scores that grow or shrink along the keys into the hundreds, or one key far above the rest: every
    kernel raises its exponent base and rescales, or never again, in each of its shares.  An fp32
    score of 128 products is off by at most 2^-17 of the sum of their sizes; weights follow it."""
    B, Hkv, page, lens = 2, 2, 32, [900, 517]
    pool = Pool(B, Hkv, page, d, lens, e4m3, seed=d + G)
    for b, L in enumerate(lens):
        for p in range(L):
            at = (int(pool.table[b, p // page]), slice(None), p % page)
            far = p if order == "rising" else L - 1 - p
            step = (8 if p == L // 2 else 1) if order == "one" else far // 64
            if e4m3:
                pool.store["ks"][at] = 119 + step if order == "one" else 114 + step
            else:
                pool.store["k"][at] = (pool.store["k"][at].float() * (step if order == "one" else 0.5 + step)).to(torch.bfloat16)
    for m in "kv":
        pool.value[m] = ref.widened(pool.store[m], pool.store[m + "s"]) if e4m3 else pool.store[m].double()
    q = (normal((B * n, G * Hkv, d), 13).float() * 3).to(torch.bfloat16)
    where, scales = pool.cuda()
    o, lse = (x.cpu().double() for x in attn.attn_paged(q.cuda(), *where, bounds([n] * B).cuda(), ints(lens).cuda(), **scales))
    ok(attn)
    wo, wl, wabs = ref.attend(q, pool.value["k"], pool.value["v"], pool.table, bounds([n] * B), lens, d ** -0.5)
    u, size = 2.0 ** -8, 0.0
    for b, L in enumerate(lens):
        k = ref.gathered(pool.value["k"], pool.table[b], L).abs().repeat_interleave(G, 0)
        size = max(size, float(torch.einsum("thd,hkd->thk", q[b * n:(b + 1) * n].double().abs(), k).max()) * d ** -0.5)
    s = 2.0 ** -17 * size
    assert bool(((o - wo).abs() <= (u + 2e-4 + 2 * s) * wabs + u * wo.abs() + 1e-6).all())
    # beside the scores' error: exp2 and log2 by a few 2^-22, and the 2^-24 of a value of wl's size
    assert float(((lse - wl).abs() - 2.0 ** -22 * wl.abs()).max()) <= s + 1e-5
    assert size < 4000


# ------------------------------------------------------------------ far addresses, broadcast views
@pytest.mark.parametrize("e4m3", [False, True])
def test_a_pool_beyond_32_bit_offsets(attn, e4m3):  # noqa: F811
    """Pages on both sides of 2^32 bytes and, for bf16, of 2^31 elements: written, read back, attended to by each
    kernel."""
    Hq, Hkv, page, d, L = 16, 8, 64, 128, 450
    room = Hkv * page * d
    pages = 2 ** 32 // (room * (1 if e4m3 else 2)) + 40
    shape = (pages, Hkv, page, d)
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kc, vc = (torch.empty(shape, dtype=dt, device="cuda") for _ in range(2))
    sc = {m: torch.empty(shape[:3], dtype=torch.uint8, device="cuda") for m in ("k_scale", "v_scale")} if e4m3 else {}
    table = ints([[pages - 1, 0, pages // 2 - 1, pages // 2, pages - 2, 3, pages - 40, pages - 41]]).cuda()
    k, v, q = (normal((L, H, d), H + i) for i, H in enumerate((Hkv, Hkv, Hq)))
    kv_len = ints([L]).cuda()
    attn.attn_cache_write(k.cuda(), v.cuda(), kc, vc, table, bounds([L]).cuda(), kv_len, **sc)
    kr, vr = attn.attn_cache_read(kc, vc, table, kv_len, N=L, **sc)
    ok(attn)
    if not e4m3:
        assert torch.equal(kr[0].transpose(0, 1).cpu(), k) and torch.equal(vr[0].transpose(0, 1).cpu(), v)
    else:
        assert float((kr[0].transpose(0, 1).cpu().double() - k.double()).abs().max()) <= 4 * 2.0 ** -4
    dense, one = (x.cpu().double() for x in (kr, vr)), torch.zeros(1, 1, dtype=torch.int32)
    dense = list(dense)
    for n in (1, 8, 40, L):
        got = attn.attn_paged(q[L - n:].cuda(), kc, vc, table, bounds([n]).cuda(), kv_len, **sc)
        ok(attn)
        check_attention(got, ref.attend(q[L - n:], *dense, one, bounds([n]), [L], d ** -0.5))
    del kc, vc, sc
    torch.cuda.empty_cache()


def test_rotation_and_read_back_beyond_2_31_elements(attn):  # noqa: F811
    """Tensors of more than 2^31 elements, compared at their two ends and around the border."""
    H, d, N = 128, 128, 2 ** 31 // (128 * 128) + 300
    x = torch.empty(1, H, N, d, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    f = attn.rope_inv_freq(d)[0]
    y, _ = attn.attn_rope(x, positions=pos, inv_freq=f)
    packed, _ = attn.attn_rope(x.reshape(N, H, d), positions=pos, inv_freq=f)
    ok(attn)
    at = torch.tensor([0, 1, N // 2, N - 301, N - 300, N - 299, N - 1])
    for h in (0, 1, H - 1):
        want = ref.rotate(x[0, h, at].cpu().unsqueeze(1), at, f.cpu(), False).squeeze(1)
        assert bool(((y[0, h, at].cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all())
        want = ref.rotate(x.reshape(N, H, d)[at, h].cpu().unsqueeze(1), at, f.cpu(), False).squeeze(1)
        assert bool(((packed[at, h].cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all())
    del y, packed, x
    B, Hkv, L, page = 64, 4, 40, 16
    pool = Pool(B, Hkv, page, d, [L] * B, False, seed=2)
    where, _ = pool.cuda()
    N = 2 ** 31 // (B * Hkv * d) + 9
    k, v = (torch.empty(B, Hkv, N, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    attn.attn_cache_read(*where, ints([L] * B).cuda(), k_out=k, v_out=v)
    ok(attn)
    for b in range(B):
        for got, n in ((k, "k"), (v, "v")):
            assert torch.equal(got[b, :, :L].cpu().double(), ref.gathered(pool.value[n], pool.table[b], L))
    del k, v
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n", [1, 20, 100])
@pytest.mark.parametrize("e4m3", [False, True])
def test_queries_broadcast_over_heads_or_tokens(attn, n, e4m3):  # noqa: F811
    """Views of stride 0, and tokens closer together than heads."""
    Hq, Hkv, d, page, L = 4, 2, 128, 64, 300
    pool = Pool(1, Hkv, page, d, [L], e4m3, seed=n)
    where, scales = pool.cuda()
    args = (*where, bounds([n]).cuda(), ints([L]).cuda())
    for q in (normal((n, 1, d), 1).cuda().expand(n, Hq, d), normal((1, Hq, d), 2).cuda().expand(n, Hq, d),
              normal((Hq, n, d), 3).cuda().transpose(0, 1)):
        got, want = attn.attn_paged(q, *args, **scales), attn.attn_paged(q.contiguous(), *args, **scales)
        ok(attn)
        assert all(torch.equal(g, w) for g, w in zip(got, want))


# ------------------------------------------------------------------ windows beyond an int, graphs that allocate
@pytest.mark.parametrize("window", [1 << 30, 1 << 31, 1 << 32, (1 << 32) + 5, (1 << 63) - 1, -(1 << 32), -(1 << 40) + 3])
def test_windows_past_32_bits_are_no_limit(attn, window):  # noqa: F811
    pool = Pool(1, 2, 32, 64, [300], False, seed=1)
    where, _ = pool.cuda()
    args = (normal((20, 4, 64), 2).cuda(), *where, bounds([20]).cuda(), ints([300]).cuda())
    want, got = attn.attn_paged(*args), attn.attn_paged(*args, window_left=window)
    ok(attn)
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("e4m3", [False, True])
def test_two_graphs_that_take_their_own_memory(attn, e4m3):  # noqa: F811
    """A decoding step and a chunk, captured without outputs or workspaces, replayed in turn while the
    lengths move: the same bits as calls outside a graph."""
    Hq, Hkv, d, page, most = 8, 2, 128, 32, 500
    pool = Pool(2, Hkv, page, d, [most, most], e4m3, seed=8)
    where, scales = pool.cuda()
    f = attn.rope_inv_freq(d)[0]
    new = normal((300, Hq + 2 * Hkv, d), 9).cuda()
    graphs = []
    for n in (1, 120):
        x, kv_len, cu = new[:2 * n].clone(), ints([n, n]).cuda(), bounds([n, n]).cuda()

        def step(x=x, kv_len=kv_len, cu=cu):
            q = attn.attn_cache_write(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], *where, cu, kv_len, **scales, inv_freq=f, q=x[:, :Hq])
            return attn.attn_paged(q, *where, cu, kv_len, **scales)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, step, kv_len, out, n))
    for at in (200, 333, 480):
        for graph, step, kv_len, out, n in graphs:
            kv_len.copy_(ints([at, at - 70]))
            graph.replay()
            got = [t.clone() for t in out]
            want = step()
            ok(attn)
            assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", FEW)
def test_wide_and_narrow_queries_in_turn_on_one_sm(attn, G, n, d):  # noqa: F811
    """700 short sequences, several to an SM, every third with a wide query: each gets the parts that it needs."""
    B, Hkv, page, L = 700, 1, 32, 20
    pool = Pool(B, Hkv, page, d, [L] * B, True, seed=G)
    codes = pool.store["k"][..., 5]
    pool.store["k"][..., 5] = torch.where(codes != 0x7f, codes & 1, codes)
    pool.value["k"] = ref.widened(pool.store["k"], pool.store["ks"])
    q = normal((B * n, G, d), 3 + G)
    wide = (torch.arange(B) % 3 == 0).repeat_interleave(n)
    q[..., 5] = torch.where(wide.unsqueeze(1), q[..., 5].float() * 2.0 ** 17, q[..., 5].float()).to(torch.bfloat16)
    where, scales = pool.cuda()
    got = attn.attn_paged(q.cuda(), *where, bounds([n] * B).cuda(), ints([L] * B).cuda(), **scales)
    ok(attn)
    check_attention(got, ref.attend(q, pool.value["k"], pool.value["v"], pool.table, bounds([n] * B), [L] * B, d ** -0.5))
