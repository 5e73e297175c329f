"""The serving operators on the GPU against plain fp64 definitions (``paged_reference``).

Tolerances, per element, from the roundings made (u = 2^-8, half a bf16 step relative to the
value; fp32 sums and functions are accounted for by the small extra terms):
- rotation: fp32 sine and cosine are off by a few 2^-24 and the angle by 2^-24 of a turn, so a
  turned value is within 1e-6 m (|a| + |b|) before the one rounding to the output's type;
- cached values: copies are exact, e4m3 codes and scale bytes follow from exact arithmetic;
- attention: P is rounded once (u), O once (u): |err| <= (u + 2e-4) sum_j w_j |v_j| + u |o| + 1e-6,
  2e-4 for the scores' fp32 sums (128 products of size up to 10, 2^-23 each) and exponentials.
"""
import math

import pytest
import torch

from tests import paged_reference as ref

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def attn():
    import __graft_entry__
    __graft_entry__.build()
    import io_aware_exact_26_b200 as a
    return a


def normal(shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def ok(attn):
    torch.cuda.synchronize()
    assert attn.attn_get_device_status() == 0


# ------------------------------------------------------------------ rotary positions
ROPE = [
    # layout, B, N, Hq, Hkv, d, rot, interleaved, dtype, far, mscale
    ("dense", 2, 5, 4, 2, 128, 128, False, torch.bfloat16, 100, 1.0),
    ("dense", 1, 257, 3, 1, 64, 64, True, torch.bfloat16, 1 << 20, 1.25),
    ("dense", 3, 33, 2, 2, 128, 32, False, torch.float32, (1 << 31) - 1, 1.0),
    ("dense", 2, 65, 5, 5, 64, 16, True, torch.float32, 1 << 24, 0.75),
    ("packed", 1, 1, 32, 8, 128, 128, False, torch.bfloat16, 4096, 1.0),
    ("packed", 1, 1001, 9, 3, 64, 48, False, torch.bfloat16, 131072, 1.0),
    ("packed", 1, 77, 7, 0, 128, 112, True, torch.float32, 1 << 30, 1.0),
]


def rope_case(case, seed=0):
    layout, B, N, Hq, Hkv, d, rot, inter, dt, far, m = case
    shape = (lambda H: (B, H, N, d)) if layout == "dense" else (lambda H: (N, H, d))
    q = normal(shape(Hq), seed + 1, dt)
    k = normal(shape(Hkv), seed + 2, dt) if Hkv else None
    g = torch.Generator().manual_seed(seed + 3)
    pos = torch.randint(-far, far, (B, N) if layout == "dense" else (N,), generator=g, dtype=torch.int64).to(torch.int32)
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return q, k, pos, f


def rope_want(x, pos, f, inter, m, inverse, layout):
    if layout == "dense":
        return ref.rotate(x.transpose(1, 2), pos, f, inter, m, inverse).transpose(1, 2)
    return ref.rotate(x, pos, f, inter, m, inverse)


def rope_bound(x, want, f, inter, m, dt):
    # |a| + |b| of a pair is at most twice the larger of the row's turned values
    size = 2 * x.double().abs()[..., :2 * f.shape[0]].amax(-1, keepdim=True)
    return 1e-6 * abs(m) * size + U[dt] * want.abs() + 1e-30


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("back", [False, True])
def test_rope_matches_the_definition(attn, case, back):
    layout, B, N, Hq, Hkv, d, rot, inter, dt, far, m = case
    q, k, pos, f = rope_case(case)
    call = attn.attn_rope_bwd if back else attn.attn_rope
    yq, yk = call(q.cuda(), k.cuda() if Hkv else None, positions=pos.cuda(), inv_freq=f.cuda(), interleaved=inter, mscale=m)
    ok(attn)
    for x, y in ((q, yq), (k, yk)):
        if x is None:
            assert y is None
            continue
        want = rope_want(x, pos, f, inter, m, back, layout)
        err = (y.cpu().double() - want).abs()
        assert bool((err <= rope_bound(x, want, f, inter, m, dt)).all()), float(err.max())
        assert torch.equal(y.cpu()[..., rot:], x[..., rot:])


def test_rope_in_place_on_views_and_one_row_of_positions(attn):
    """Slices of one fused projection (packed), and of a transposed one (dense), turned in place:
    the same bits as out of place, the neighbours untouched."""
    T, Hq, Hkv, d = 50, 6, 2, 128
    f = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d).cuda()
    pos = torch.arange(7, 7 + T, dtype=torch.int32).cuda()
    qkv = normal((T, Hq + 2 * Hkv, d), 5).cuda()
    before = qkv.clone()
    want_q, want_k = attn.attn_rope(qkv[:, :Hq].contiguous(), qkv[:, Hq:Hq + Hkv].contiguous(), positions=pos, inv_freq=f)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    attn.attn_rope(q, k, positions=pos, inv_freq=f, q_out=q, k_out=k)
    ok(attn)
    assert torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(qkv[:, Hq + Hkv:], before[:, Hq + Hkv:])
    x = normal((2, T, 4, d), 6).cuda()                    # [B, N, H, d], used as [B, H, N, d]
    y, _ = attn.attn_rope(x.transpose(1, 2), positions=pos, inv_freq=f)
    z, _ = attn.attn_rope(x.transpose(1, 2).contiguous(), positions=pos.expand(2, T).contiguous(), inv_freq=f)
    ok(attn)
    assert torch.equal(y, z)


def test_rope_gradient_matches_differences(attn):
    """d/dx sum(g * rope(x)) along random directions, in fp32: the operator is linear, so the
    central difference has no truncation error; both sides carry fp32 rounding only."""
    case = ("dense", 2, 19, 3, 1, 64, 48, True, torch.float32, 5000, 1.3)
    q, k, pos, f = rope_case(case, seed=40)
    pos, f = pos.cuda(), f.cuda()
    args = dict(positions=pos, inv_freq=f, interleaved=True, mscale=1.3)
    gq, gk = normal(q.shape, 50, torch.float32).cuda(), normal(k.shape, 51, torch.float32).cuda()
    dq, dk = attn.attn_rope_bwd(gq, gk, **args)
    for seed in range(3):
        hq, hk = normal(q.shape, 60 + seed, torch.float32).cuda(), normal(k.shape, 70 + seed, torch.float32).cuda()
        up, dn = (attn.attn_rope(q.cuda() + s * hq, k.cuda() + s * hk, **args) for s in (1.0, -1.0))
        diff = sum(float((g.double() * (u.double() - d.double())).sum()) / 2 for g, u, d in zip((gq, gk), up, dn))
        form = float((dq.double() * hq.double()).sum() + (dk.double() * hk.double()).sum())
        scale = float((gq.double().abs() * hq.double().abs()).sum() + (gk.double().abs() * hk.double().abs()).sum())
        assert abs(diff - form) <= 1e-5 * scale
    ok(attn)


# ------------------------------------------------------------------ pool and sequences
class Pool:
    """A page pool on the CPU (fp64 values and the stored form), pages in random order, every
    byte that no sequence owns set to NaN."""

    def __init__(self, B, Hkv, page, d, lens, e4m3, seed, room=3, fill=True):
        g = torch.Generator().manual_seed(seed)
        need = [-(-max(0, L) // page) for L in lens]
        self.pages, self.page, self.e4m3 = sum(need) + room, page, e4m3
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((B, max(need + [1]) + 1), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.pages, Hkv, page, d)
        self.store, self.value = {}, {}
        for i, n in enumerate("kv"):
            x = torch.randn(shape, generator=g)
            if e4m3:
                self.store[n] = x.mul(20).to(torch.float8_e4m3fn).view(torch.uint8)
                self.store[n + "s"] = torch.randint(119, 124, shape[:3], generator=g).to(torch.uint8)
            else:
                self.store[n] = x.to(torch.bfloat16)
        if not fill:
            for n in self.store:
                self.store[n].zero_()
        own = torch.zeros(shape[:3], dtype=torch.bool)
        for b, L in enumerate(lens):
            for p in range(max(0, L)):
                own[self.table[b, p // page].long(), :, p % page] = True
        for n in "kv":
            if e4m3:
                self.store[n][~own] = 0x7f
            else:
                self.store[n][~own] = math.nan
            self.value[n] = ref.widened(self.store[n], self.store[n + "s"]) if e4m3 else self.store[n].double()

    def cuda(self):
        k, v = (self.store[n].cuda() for n in "kv")
        if self.e4m3:
            return (k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), self.table.cuda()), dict(
                k_scale=self.store["ks"].cuda(), v_scale=self.store["vs"].cuda())
        return (k, v, self.table.cuda()), {}


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


def bounds(new):
    return ints([0] + torch.tensor(new).cumsum(0).tolist())


# ------------------------------------------------------------------ cache write and read
WRITE = [
    # Hkv, Hq, d, page, e4m3, rot, interleaved, new, len
    (2, 0, 128, 16, False, 0, False, [1, 1, 1], [1, 17, 300]),
    (1, 4, 64, 64, False, 64, False, [5, 0, 40], [5, 90, 41]),
    (8, 8, 128, 32, False, 32, True, [33], [100]),
    (3, 0, 64, 16, True, 0, False, [7, 0, 1, 65], [7, 3, 50, 130]),
    (2, 6, 128, 256, True, 128, False, [1, 30], [300, 31]),
    (4, 4, 64, 128, True, 48, True, [50, 2], [50, 200]),
]


@pytest.mark.parametrize("case", WRITE, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("checks", [False, True])
def test_cache_write_puts_every_row_in_its_place(attn, case, checks):
    Hkv, Hq, d, page, e4m3, rot, inter, new, lens = case
    T, B = sum(new), len(new)
    pad = 3                                               # rows behind the last sequence
    qkv = normal((T + pad, Hq + 2 * Hkv, d), T + d)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pool = Pool(B, Hkv, page, d, lens, e4m3, seed=page)
    (kc, vc, table), scales = pool.cuda()
    cu, kv_len = bounds(new), ints(lens)
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) if rot else None
    gq = qkv.cuda()
    kw = dict(inv_freq=f.cuda(), interleaved=inter, mscale=1.2) if rot else {}
    q_out = torch.full((T + pad, Hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    if Hq:
        kw.update(q=gq[:, :Hq], q_out=q_out)
    import contextlib
    with attn.use_library(attn.checks_library_path) if checks else contextlib.nullcontext():
        attn.attn_cache_write(gq[:, Hq:Hq + Hkv], gq[:, Hq + Hkv:], kc, vc, table, cu.cuda(), kv_len.cuda(), **scales, **kw)
        ok(attn)
    pos = torch.cat([torch.arange(L - n, L) for n, L in zip(new, lens)])
    turned = (lambda x: ref.rotate(x[:T], pos, f, inter, 1.2)) if rot else (lambda x: x[:T].double())
    if Hq:
        want = turned(q)
        err = (q_out.cpu()[:T].double() - want).abs()
        assert bool((err <= rope_bound(q[:T], want, f, inter, 1.2, torch.bfloat16)).all())
        assert bool((q_out[T:] == 9.0).all())
    touched = torch.zeros(kc.shape[:3], dtype=torch.bool)
    t = 0
    for b, (n, L) in enumerate(zip(new, lens)):
        for p in range(L - n, L):
            at = (int(pool.table[b, p // page]), slice(None), p % page)
            touched[at] = True
            for name, got, x in (("k", kc, turned(k)[t]), ("v", vc, v[t].double())):
                if not e4m3:
                    y = got[at].cpu().double()
                    lim = rope_bound(k[t], x, f, inter, 1.2, torch.bfloat16) if name == "k" and rot else torch.zeros(())
                    assert bool(((y - x).abs() <= lim).all())
                    continue
                codes = got.view(torch.uint8)[at].cpu()
                byte = scales[name + "_scale"][at].cpu()
                for h in range(Hkv):
                    wc, wb = ref.quantise_row(x[h])
                    if name == "v" or not rot:
                        assert codes[h].tolist() == wc and int(byte[h]) == wb
                    else:
                        # rotated in fp32 (1e-6): a value next to a rounding border may go to either
                        # side, so a code is off by half a step and that error at most
                        unit = 2.0 ** (int(byte[h]) - 127)
                        y = ref.widened(codes[h], byte[h])
                        step = torch.exp2(torch.floor(torch.log2((x[h].abs() / unit).clamp_min(2.0 ** -6))) - 3) * unit
                        assert abs(int(byte[h]) - wb) <= 1
                        assert bool(((y - x[h]).abs() <= step * (0.5 + 1e-3) + 1e-5).all())
            t += 1
    for name, got in (("k", kc), ("v", vc)):              # rows that no token maps to
        a, w = (got.view(torch.uint8) if e4m3 else got.view(torch.int16)).cpu(), pool.store[name]
        w = w if e4m3 else w.view(torch.int16)
        assert torch.equal(a[~touched], w[~touched])
        if e4m3:
            assert torch.equal(scales[name + "_scale"].cpu()[~touched], pool.store[name + "s"][~touched])


def test_cache_write_scales_at_the_borders(attn):
    """Rows whose maximum sits on, just above and below a power-of-two border, zeros, subnormals, the
    largest values, infinities and NaN: codes and bytes from the definition."""
    tops = [448.0, 450.0, 446.0, 1.75, 1.7578125, 0.875, 0.0, 2.0 ** -126, 2.0 ** -133, 3.3895313892515355e38,
            57344.0, 57600.0, 1e-38, 1.0]
    rows = []
    for i, a in enumerate(tops):
        r = normal((64,), 900 + i, torch.float32).clamp(-3.5, 3.5) / 4 * a
        r[i] = a if i % 2 else -a
        rows.append(r.to(torch.bfloat16))
    for bad in (math.inf, -math.inf, math.nan):
        r = normal((64,), 7, torch.bfloat16)
        r[5] = bad
        rows.append(r)
    x = torch.stack(rows).unsqueeze(1)                     # [T, 1, 64]
    T = x.shape[0]
    kc, vc = (torch.zeros(3, 1, 16, 64, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(3, 1, 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = ints([[2, 0, 1]]).cuda()
    attn.attn_cache_write(x.cuda(), x.cuda(), kc, vc, table, bounds([T]).cuda(), ints([T]).cuda(), k_scale=ks, v_scale=vs)
    kr, vr = attn.attn_cache_read(kc, vc, table, ints([T]).cuda(), k_scale=ks, v_scale=vs, N=T + 2)
    ok(attn)
    for t in range(T):
        codes, byte = ref.quantise_row(x[t, 0])
        page = (2, 0, 1)[t // 16]
        assert kc.view(torch.uint8)[page, 0, t % 16].tolist() == codes, t
        assert int(ks[page, 0, t % 16]) == byte, t
    assert torch.equal(kc.view(torch.uint8), vc.view(torch.uint8)) and torch.equal(ks, vs)
    assert bool((kr[0, 0, T:] == 0).all()) and torch.equal(kr.view(torch.int16), vr.view(torch.int16))


@pytest.mark.parametrize("d", [64, 128])
def test_cache_read_widens_every_code_under_every_scale(attn, d):
    """All 256 codes under the 248 scale bytes that the write produces: the bf16 nearest to
    code * 2^(byte - 127), which is that value itself unless bf16 cannot hold it."""
    byte = torch.arange(248, dtype=torch.uint8).repeat_interleave(256 // d)
    L = byte.numel()
    codes = torch.arange(256, dtype=torch.uint8).reshape(256 // d, d).repeat(248, 1)
    pages = -(-L // 256)
    c = torch.zeros(pages * 256, d, dtype=torch.uint8)
    s = torch.zeros(pages * 256, dtype=torch.uint8)
    c[:L], s[:L] = codes, byte
    kc = c.reshape(pages, 1, 256, d).cuda().view(torch.float8_e4m3fn)
    vc = kc.view(torch.uint8).flip(-1).contiguous().view(torch.float8_e4m3fn)
    ks = s.reshape(pages, 1, 256).cuda()
    table = torch.arange(pages, dtype=torch.int32).reshape(1, pages).cuda()
    k, v = attn.attn_cache_read(kc, vc, table, ints([L]).cuda(), k_scale=ks, v_scale=ks, N=L)
    ok(attn)
    want = ref.widened(codes, byte).to(torch.float32).to(torch.bfloat16)      # fp32 holds all of them
    for got, w in ((k, want), (v, want.flip(-1))):
        got = got[0, 0].cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(w))
        assert torch.equal(got.nan_to_num(0.0), w.nan_to_num(0.0))
        assert torch.equal(torch.signbit(got) & (got == 0), torch.signbit(w) & (w == 0))


@pytest.mark.parametrize("page,d,e4m3,lens,N", [(16, 64, False, [0, 1, 33, 200], 64), (64, 128, False, [130, 64], 140),
                                                (256, 128, True, [300, 5], 300), (32, 64, True, [97, 0, 31], 97)])
def test_cache_read_gathers_what_is_there(attn, page, d, e4m3, lens, N):
    pool = Pool(len(lens), 3, page, d, lens, e4m3, seed=N)
    where, scales = pool.cuda()
    k_out, v_out = (torch.full((len(lens), 3, N, d), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for lib in (attn.library_path, attn.checks_library_path):
        with attn.use_library(lib):
            attn.attn_cache_read(*where, ints(lens).cuda(), **scales, k_out=k_out, v_out=v_out)
            ok(attn)
    for b, L in enumerate(lens):
        L = min(L, N)
        for got, n in ((k_out, "k"), (v_out, "v")):
            want = ref.gathered(pool.value[n], pool.table[b], L)
            assert torch.equal(got[b, :, :L].cpu().double(), want)
            assert bool((got[b, :, L:] == 5.0).all())


# ------------------------------------------------------------------ attention
PAGED = [
    # Hq, Hkv, d, page, e4m3, new, len, causal, window
    (1, 1, 128, 16, False, [1], [1], True, None),
    (8, 2, 128, 64, False, [1, 1, 1], [1000, 129, 128], True, None),
    (8, 8, 64, 32, False, [1, 0, 1], [77, 500, 300], True, None),
    (16, 1, 128, 128, False, [1], [2500], True, None),
    (128, 1, 64, 64, False, [1, 2], [200, 131], True, None),
    (10, 2, 64, 16, False, [3, 60, 1], [500, 60, 127], True, None),
    (6, 2, 128, 256, False, [130, 5], [400, 300], True, None),
    (4, 4, 128, 64, False, [200], [200], True, None),
    (4, 2, 64, 128, False, [150, 1], [290, 700], True, 100),
    (4, 1, 128, 16, False, [70, 1], [333, 600], True, 0),
    (4, 2, 128, 32, False, [20, 3], [150, 260], False, None),
    (4, 2, 64, 64, False, [20, 3], [150, 260], False, 30),
    (8, 2, 128, 16, True, [1, 1, 1], [1000, 16, 130], True, None),
    (8, 4, 64, 64, True, [1, 90], [400, 333], True, None),
    (5, 1, 128, 128, True, [40, 1], [100, 513], True, 64),
    (8, 8, 64, 256, True, [140, 2], [140, 259], True, None),
    (2, 2, 128, 32, True, [9], [70], False, None),
    (3, 1, 64, 64, False, [5, 4, 2], [3, 0, 2], True, None),     # more new tokens than keys: empty rows
    (3, 1, 64, 64, True, [5, 4, 2], [3, 0, 2], True, None),
]


def check_attention(got, want):
    o, lse = (x.cpu().double() for x in got)
    wo, wl, wabs = want
    u = U[torch.bfloat16]
    err = (o - wo).abs()
    bound = (u + 2e-4) * wabs + u * wo.abs() + 1e-6
    assert bool((err <= bound).all()), (float((err - bound).max()), int((err > bound).sum()))
    empty = torch.isinf(wl)
    assert torch.equal(torch.isinf(lse), empty) and bool((o[empty] == 0).all())
    assert float((lse - wl)[~empty].abs().max() if bool((~empty).any()) else 0.0) <= 1e-3


def run_paged(attn, case, seed, checks=False, workspace=None):
    Hq, Hkv, d, page, e4m3, new, lens, causal, window = case
    T, B, pad = sum(new), len(new), 2
    pool = Pool(B, Hkv, page, d, lens, e4m3, seed=seed)
    where, scales = pool.cuda()
    wide = normal((T + pad, Hq + 3, d), seed + 1)          # a strided view of a wider projection
    q = wide[:, 1:1 + Hq]
    o = torch.full((T + pad, Hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + pad, Hq), 3.0, device="cuda")
    import contextlib
    with attn.use_library(attn.checks_library_path) if checks else contextlib.nullcontext():
        attn.attn_paged(wide.cuda()[:, 1:1 + Hq], *where, bounds(new).cuda(), ints(lens).cuda(), **scales, o=o, lse=lse,
                        causal=causal, window_left=window, workspace=workspace)
        ok(attn)
    assert bool((o[T:] == 3.0).all()) and bool((lse[T:] == 3.0).all())
    want = ref.attend(q[:T], pool.value["k"], pool.value["v"], pool.table, bounds(new), lens, d ** -0.5, causal, window)
    return (o[:T], lse[:T]), want


@pytest.mark.parametrize("case", PAGED, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("checks", [True, False])
def test_paged_attention_matches_the_definition(attn, case, checks):
    check_attention(*run_paged(attn, case, seed=sum(case[5]) + case[2], checks=checks))


def ragged(B, seed, most=90):
    """Ragged batch whose tiles outnumber the SMs several times, so that every CTA works on several
    items of very different row counts, one after the other."""
    g = torch.Generator().manual_seed(seed)
    new = [int(n) for n in torch.randint(0, most, (B,), generator=g)]
    new[1::3] = [1] * len(new[1::3])
    return new, [n + int(x) for n, x in zip(new, torch.randint(0, 700, (B,), generator=g))]


@pytest.mark.parametrize("Hq,Hkv,d,page,e4m3,window", [(8, 8, 64, 16, False, None), (12, 4, 128, 64, False, 200),
                                                       (16, 16, 128, 32, True, None), (20, 4, 64, 128, True, 77)])
def test_paged_attention_of_many_ragged_items(attn, Hq, Hkv, d, page, e4m3, window):
    new, lens = ragged(48, seed=Hq + d)
    check_attention(*run_paged(attn, (Hq, Hkv, d, page, e4m3, new, lens, True, window), seed=d))


@pytest.mark.parametrize("Hq,Hkv,d,page,e4m3,window", [(8, 2, 128, 64, False, None), (6, 2, 64, 16, False, 150),
                                                       (4, 4, 128, 128, False, None), (5, 1, 64, 32, True, None),
                                                       (6, 2, 128, 16, True, None), (8, 8, 128, 64, True, 300)])
def test_paged_attention_of_ragged_chunks(attn, Hq, Hkv, d, page, e4m3, window):
    """Chunks of up to several query tiles beside single tokens and empty ones."""
    new, lens = ragged(20, seed=Hq * d, most=420)
    check_attention(*run_paged(attn, (Hq, Hkv, d, page, e4m3, new, lens, True, window), seed=d))


@pytest.mark.parametrize("rows", [3, 4, 5, 8, 9, 16, 17, 32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
def test_paged_attention_around_each_row_count_of_a_kernel(attn, rows, d, e4m3):
    """The mean of rows per sequence picks the kernel: just at, below and above each step, with a
    sequence of many times the mean in it, one of no token, and one query head to a cache head."""
    new, lens = [rows, 0, 4 * rows - 2, 1, 1], [300, 40, 190, 129, 1]
    new[0] = 5 * rows - sum(new[1:])                                  # mean of exactly `rows`
    check_attention(*run_paged(attn, (2, 2, d, 32, e4m3, new, lens, True, None), seed=rows * d))


@pytest.mark.parametrize("Hq", [4, 8, 12, 32, 64])
@pytest.mark.parametrize("e4m3", [False, True])
def test_paged_attention_is_repeatable(attn, Hq, e4m3):
    """Every form of the kernel, many pieces per SM: 40 launches in a row give the same bits."""
    B, Hkv, d, page, L = 24, 2, 64 if e4m3 else 128, 16, 3000
    lens = [L - 57 * b for b in range(B)]
    pool = Pool(B, Hkv, page, d, lens, e4m3, seed=Hq)
    where, scales = pool.cuda()
    new = [1 + 3 * (b % 2) if Hq < 64 else 4 for b in range(B)]
    q = normal((sum(new), Hq, d), Hq).cuda()
    args = (q, *where, bounds(new).cuda(), ints(lens).cuda())
    o, lse = attn.attn_paged(*args, **scales)
    again = [attn.attn_paged(*args, **scales) for _ in range(40)]
    ok(attn)
    assert all(torch.equal(a, o) and torch.equal(b, lse) for a, b in again)


@pytest.mark.parametrize("e4m3", [False, True])
def test_paged_attention_over_a_long_context_in_many_parts(attn, e4m3):
    """One KV head, one token: a single row of 160 key tiles is shared out over all SMs and merged;
    stale workspace contents do not matter, equal calls give equal bits."""
    case = (4, 1, 128, 64, e4m3, [1], [20400], True, None)
    size = attn.attn_paged_workspace_size(3, 1, 4, 1, 128)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    got, want = run_paged(attn, case, seed=3, workspace=ws)
    check_attention(got, want)
    again, _ = run_paged(attn, case, seed=3)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_paged_attention_of_large_scores_and_dominant_keys(attn):
    """Scores of both signs in the hundreds, maxima that rise tile by tile: the running rescale."""
    Hq, Hkv, d, page, L = 4, 2, 128, 64, 900
    pool = Pool(1, Hkv, page, d, [L], False, seed=12)
    ramp = torch.linspace(0.5, 12, L)
    for p in range(L):
        at = (int(pool.table[0, p // page]), slice(None), p % page)
        pool.store["k"][at] = (pool.store["k"][at].float() * ramp[p]).to(torch.bfloat16)
    pool.value["k"] = pool.store["k"].double()
    q = (normal((30, Hq, d), 13).float() * 4).to(torch.bfloat16)
    where, _ = pool.cuda()
    got = attn.attn_paged(q.cuda(), *where, bounds([30]).cuda(), ints([L]).cuda())
    ok(attn)
    wo, wl, wabs = ref.attend(q, pool.value["k"], pool.value["v"], pool.table, bounds([30]), [L], d ** -0.5)
    # scores up to ~600: an fp32 score is off by up to 128 * 2^-24 * sum|q k| * scale ~ 600 * 4 * 2^-17
    # (the products' sizes add up to about 4 times the largest score) = 0.02 at worst, so weights by 2%
    u, s = U[torch.bfloat16], 0.02
    err = (got[0].cpu().double() - wo).abs()
    assert bool((err <= (u + 2 * s) * wabs + u * wo.abs() + 1e-6).all())
    assert float((got[1].cpu().double() - wl).abs().max()) <= s


def test_paged_attention_agrees_with_the_dense_decode(attn):
    """A batch of equal lengths, gathered by attn_cache_read and given to attn_decode."""
    B, Hq, Hkv, L, d, page = 3, 8, 2, 700, 128, 32
    pool = Pool(B, Hkv, page, d, [L] * B, False, seed=8)
    where, _ = pool.cuda()
    q = normal((B, Hq, d), 9).cuda()
    o, lse = attn.attn_paged(q, *where, bounds([1] * B).cuda(), ints([L] * B).cuda())
    k, v = attn.attn_cache_read(*where, ints([L] * B).cuda(), N=L)
    o2, l2 = attn.attn_decode(q.reshape(B, Hq, 1, d), k, v, causal=True)
    ok(attn)
    assert float((lse - l2.reshape(B, Hq)).abs().max()) <= 1e-4
    assert float((o.float() - o2.reshape(B, Hq, d).float()).abs().max()) <= 2 * U[torch.bfloat16]


def test_paged_cache_interleaved_page_by_page(attn):
    """K and V as halves of one [pages, 2, Hkv, page, d] buffer: the page stride is followed by the
    write, the read and the attention."""
    Hkv, page, d, L = 2, 16, 64, 50
    both = torch.full((9, 2, Hkv, page, d), math.nan, dtype=torch.bfloat16, device="cuda")
    kc, vc = both[:, 0], both[:, 1]
    table = ints([[7, 2, 4, 0]]).cuda()
    k, v, q = (normal((L, H, d), 20 + H) for H in (Hkv, Hkv, 4))
    cu, kv_len = bounds([L]).cuda(), ints([L]).cuda()
    attn.attn_cache_write(k.cuda(), v.cuda(), kc, vc, table, cu, kv_len)
    kr, vr = attn.attn_cache_read(kc, vc, table, kv_len, N=L)
    got = attn.attn_paged(q.cuda(), kc, vc, table, cu, kv_len)
    ok(attn)
    assert torch.equal(kr[0].transpose(0, 1).cpu(), k) and torch.equal(vr[0].transpose(0, 1).cpu(), v)
    dense = k.double().transpose(0, 1).unsqueeze(0), v.double().transpose(0, 1).unsqueeze(0)     # one page of L rows
    check_attention(got, ref.attend(q, *dense, torch.zeros(1, 1, dtype=torch.int32), bounds([L]), [L], d ** -0.5))


def test_window_does_not_read_evicted_pages(attn):
    """Table entries of pages wholly before every row's window may be invalid: nothing is recorded,
    and NaN in the positions before the window does not reach the result."""
    Hq, Hkv, d, page, L, window = 4, 2, 64, 16, 300, 40
    pool = Pool(1, Hkv, page, d, [L], False, seed=31)
    first = L - 1 - window
    for p in range(first):
        at = (int(pool.table[0, p // page]), slice(None), p % page)
        for n in "kv":
            pool.store[n][at] = math.nan
            pool.value[n][at] = 0.0
    table = pool.table.clone()
    table[0, :first // page] = 1 << 30
    (kc, vc, _), _ = pool.cuda()
    q = normal((1, Hq, d), 32)
    got = attn.attn_paged(q.cuda(), kc, vc, table.cuda(), bounds([1]).cuda(), ints([L]).cuda(), window_left=window)
    ok(attn)
    check_attention(got, ref.attend(q, pool.value["k"], pool.value["v"], pool.table, bounds([1]), [L], d ** -0.5, True, window))


def test_bad_pages_are_reported_and_never_followed(attn):
    """Entries outside the pool and positions behind the table: writes skipped, reads zero, the other
    sequence unharmed, the status reported once."""
    BAD = -10
    Hkv, page, d = 2, 16, 64
    kc, vc = (torch.full((4, Hkv, page, d), 2.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = ints([[4, 1], [2, 3], [-1, 9999999]]).cuda()
    cu, kv_len = bounds([20, 20, 1]).cuda(), ints([20, 40, 20]).cuda()     # sequence 1 passes its two pages
    k, v = normal((41, Hkv, d), 1).cuda(), normal((41, Hkv, d), 2).cuda()
    attn.attn_cache_write(k, v, kc, vc, table, cu, kv_len)
    assert attn.attn_get_device_status() == BAD and attn.attn_get_device_status() == 0
    assert bool((kc[0] == 2.0).all())
    assert torch.equal(kc[1, :, :4].transpose(0, 1), k[16:20]) and bool((kc[1, :, 4:] == 2.0).all())
    assert torch.equal(kc[3, :, 4:].transpose(0, 1), k[20:32]) and bool((kc[3, :, :4] == 2.0).all())
    kr, _ = attn.attn_cache_read(kc, vc, table, kv_len, N=40)
    assert attn.attn_get_device_status() == BAD
    assert bool((kr[0, :, :16] == 0).all()) and torch.equal(kr[0, :, 16:20].transpose(0, 1), k[16:20])
    assert bool((kr[2, :, :20] == 0).all())
    q = normal((41, 4, d), 3).cuda()
    good, gl = attn.attn_paged(q[:1], kc, vc, ints([[2, 3]]).cuda(), ints([0, 1]).cuda(), ints([32]).cuda())
    ok(attn)
    o, lse = attn.attn_paged(q[:2], kc, vc, ints([[2, 3], [4, -5]]).cuda(), ints([0, 1, 2]).cuda(), ints([32, 20]).cuda())
    assert attn.attn_get_device_status() == BAD
    assert torch.equal(o[0], good[0]) and torch.equal(lse[0], gl[0])
    assert bool((o[1] == 0).all()) and float((lse[1] - math.log(20)).abs().max()) <= 1e-5    # zero K and V
    ok(attn)


def test_lengths_beyond_the_table_are_reported_and_bounded(attn):
    """A kv_len far past the table: the call ends at once, reports it, and leaves the other sequence's
    result as it is alone."""
    pool = Pool(1, 2, 16, 64, [30], False, seed=4)
    (kc, vc, table), _ = pool.cuda()
    q = normal((2, 4, 64), 5).cuda()
    alone = attn.attn_paged(q[:1], kc, vc, table, ints([0, 1]).cuda(), ints([30]).cuda())
    ok(attn)
    both = table.repeat(2, 1).contiguous()
    o, lse = attn.attn_paged(q, kc, vc, both, ints([0, 1, 2]).cuda(), ints([30, 1 << 29]).cuda())
    assert attn.attn_get_device_status() == -10
    assert torch.equal(o[0], alone[0][0]) and torch.equal(lse[0], alone[1][0])
    ok(attn)


@pytest.mark.parametrize("e4m3", [False, True])
def test_sparse_batches_and_rows_that_belong_to_nobody(attn, e4m3):
    """200 slots of which a few have tokens, packed rows that begin behind row 0: written, attended, and
    every other row left alone."""
    B, Hq, Hkv, d, page, first = 200, 4, 2, 64, 32, 3
    new, lens = [0] * B, [0] * B
    for b, n in ((0, 1), (37, 5), (38, 1), (120, 40), (199, 2)):
        new[b], lens[b] = n, n + 90 + b
    T = sum(new)
    pool = Pool(B, Hkv, page, d, lens, e4m3, seed=2)
    (kc, vc, table), scales = pool.cuda()
    cu = bounds(new) + first
    rows = normal((first + T + 2, Hq + 2 * Hkv, d), 6)
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    attn.attn_cache_write(k.cuda(), v.cuda(), kc, vc, table, cu.cuda(), ints(lens).cuda(), **scales)
    o = torch.full((first + T + 2, Hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((first + T + 2, Hq), 3.0, device="cuda")
    attn.attn_paged(q.cuda(), kc, vc, table, cu.cuda(), ints(lens).cuda(), **scales, o=o, lse=lse)
    ok(attn)
    outside = torch.ones(first + T + 2, dtype=torch.bool)
    outside[first:first + T] = False
    assert bool((o.cpu()[outside] == 3.0).all()) and bool((lse.cpu()[outside] == 3.0).all())
    owned = torch.zeros(kc.shape[:3], dtype=torch.bool)
    for b, L in enumerate(lens):
        for p in range(L):
            owned[int(table[b, p // page]), :, p % page] = True
    if e4m3:
        kv = [ref.widened(c.view(torch.uint8).cpu(), s.cpu()) for c, s in ((kc, scales["k_scale"]), (vc, scales["v_scale"]))]
    else:
        kv = [c.cpu().double() for c in (kc, vc)]
    for c, n in zip(kv, "kv"):
        stored = pool.value[n]
        assert bool((c[~owned].isnan() == stored[~owned].isnan()).all())       # nothing written elsewhere
    want = ref.attend(q[first:first + T], *kv, pool.table, bounds(new), lens, d ** -0.5)
    check_attention((o[first:first + T], lse[first:first + T]), want)


@pytest.mark.parametrize("T,Hq", [(1, 4), (1, 40), (30, 8), (200, 8)])
def test_scale_zero_attends_uniformly_even_to_zero_rows(attn, T, Hq):
    """scale = 0 over an e4m3 cache of zero rows under the smallest scale, and over a bf16 one."""
    Hkv, page, d, L = 4, 16, 64, 333
    for dt in (torch.float8_e4m3fn, torch.bfloat16):
        kc = torch.zeros(21, Hkv, page, d, dtype=dt, device="cuda")
        vc = torch.full((21, Hkv, page, d), 2.0, device="cuda").to(dt)
        sc = dict(k_scale=torch.zeros(21, Hkv, page, dtype=torch.uint8, device="cuda"),
                  v_scale=torch.full((21, Hkv, page), 127, dtype=torch.uint8, device="cuda")) if dt != torch.bfloat16 else {}
        table = torch.arange(21, dtype=torch.int32).reshape(1, 21).cuda()
        o, lse = attn.attn_paged(normal((T, Hq, d), 1).cuda(), kc, vc, table, bounds([T]).cuda(), ints([L]).cuda(), **sc,
                                 scale=0.0, causal=False, window_left=(1 << 31) - 1)
        ok(attn)
        # Every score is 0 and every term of the sum 1.  Rows beyond one tile (bf16) take 2 of 8 pairs
        # of terms at d = 64 from a cubic with a relative error of up to 7.5e-5 (its constant term is
        # 7.2e-5 below 1), so the sum is off by at most 2/8 * 7.5e-5 = 1.9e-5, and its logarithm too.
        assert bool((o == 2.0).all()) and float((lse - math.log(L)).abs().max()) <= 1e-5 + 2 / 8 * 7.5e-5


def test_calls_on_two_streams_with_a_workspace_each(attn):
    """Two batches at once on two streams give what they give alone."""
    out = []
    for seed, lens in ((1, [3000, 40]), (2, [900, 2200])):
        pool = Pool(2, 2, 32, 128, lens, False, seed=seed)
        where, _ = pool.cuda()
        q = normal((2, 8, 128), seed).cuda()
        args = (q, *where, bounds([1, 1]).cuda(), ints(lens).cuda())
        ws = torch.empty(attn.attn_paged_workspace_size(2, 2, 8, 2, 128), dtype=torch.uint8, device="cuda")
        out.append((args, ws, attn.attn_paged(*args, workspace=ws), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (args, ws, _, s) in enumerate(out):
            got[i].append(attn.attn_paged(*args, workspace=ws, stream=s))
    ok(attn)
    for i, (_, _, want, _) in enumerate(out):
        for o, lse in got[i]:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_a_captured_step_follows_growing_lengths(attn):
    """Rotate, write and attend as one decoding step, captured once and replayed while kv_len, the
    table and the new rows change in place; every step against the definition."""
    B, Hq, Hkv, d, page, e4m3 = 3, 6, 2, 128, 16, False
    lens = [14, 40, 127]
    steps = 5
    pool = Pool(B, Hkv, page, d, [L + steps for L in lens], e4m3, seed=77)
    (kc, vc, table), _ = pool.cuda()
    f = attn.rope_inv_freq(64)[0]
    x = torch.zeros(B, Hq + 2 * Hkv, d, dtype=torch.bfloat16, device="cuda")
    kv_len, cu = ints(lens).cuda(), bounds([1] * B).cuda()
    q_out = torch.zeros(B, Hq, d, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.zeros_like(q_out), torch.zeros(B, Hq, device="cuda")
    ws = torch.empty(attn.attn_paged_workspace_size(B, B, Hq, Hkv, d), dtype=torch.uint8, device="cuda")

    def step():
        attn.attn_cache_write(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, table, cu, kv_len, inv_freq=f, q=x[:, :Hq],
                              q_out=q_out)
        attn.attn_paged(q_out, kc, vc, table, cu, kv_len, o=o, lse=lse, workspace=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    now = [L for L in lens]
    for i in range(steps):
        now = [L + 1 for L in now]
        new = normal((B, Hq + 2 * Hkv, d), 500 + i)
        x.copy_(new)
        kv_len.copy_(ints(now))
        graph.replay()
        ok(attn)
        pos = torch.tensor(now) - 1
        for b in range(B):
            at = (int(pool.table[b, (now[b] - 1) // page]), slice(None), (now[b] - 1) % page)
            kt = ref.rotate(new[b:b + 1, Hq:Hq + Hkv], pos[b:b + 1], f.cpu(), False)[0]
            assert bool(((kc[at].cpu().double() - kt).abs() <= U[torch.bfloat16] * kt.abs() + 1e-5).all())
            assert torch.equal(vc[at].cpu(), new[b, Hq + Hkv:])
        check_attention((o, lse), ref.attend(q_out.cpu(), kc.cpu().double(), vc.cpu().double(), pool.table, bounds([1] * B),
                                             now, d ** -0.5))


def test_a_prompt_in_chunks_equals_the_dense_causal_forward(attn):
    """A prompt written and attended in ragged chunks, 8-bit and bf16 caches; the bf16 rows agree with
    attn_fwd on the whole prompt."""
    N, Hq, Hkv, d, page = 500, 8, 4, 64, 32
    q, k, v = (normal((N, H, d), 80 + H) for H in (Hq, Hkv, Hkv))
    table = torch.randperm(20, generator=torch.Generator().manual_seed(1))[:16].to(torch.int32).reshape(1, 16).cuda()
    want, wl = attn.attn_fwd(*(x.transpose(0, 1).unsqueeze(0).contiguous().cuda() for x in (q, k, v)), causal=True)
    for e4m3 in (False, True):
        dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        kc, vc = (torch.zeros(20, Hkv, page, d, dtype=dt, device="cuda") for _ in range(2))
        sc = dict(k_scale=torch.zeros(20, Hkv, page, dtype=torch.uint8, device="cuda"),
                  v_scale=torch.zeros(20, Hkv, page, dtype=torch.uint8, device="cuda")) if e4m3 else {}
        at, o, lse = 0, [], []
        for n in (1, 130, 17, 300, 52):
            cu, kv_len = bounds([n]).cuda(), ints([at + n]).cuda()
            part = slice(at, at + n)
            attn.attn_cache_write(k[part].cuda(), v[part].cuda(), kc, vc, table, cu, kv_len, **sc)
            a, b = attn.attn_paged(q[part].cuda(), kc, vc, table, cu, kv_len, **sc)
            o.append(a)
            lse.append(b)
            at += n
        kr, vr = attn.attn_cache_read(kc, vc, table, ints([N]).cuda(), N=N, **sc)
        ok(attn)
        got = torch.cat(o), torch.cat(lse)
        check_attention(got, ref.attend(q, kr.cpu().double(), vr.cpu().double(), torch.zeros(1, 1, dtype=torch.int32),
                                        bounds([N]), [N], d ** -0.5))
        if not e4m3:
            assert float((got[1] - wl[0].T).abs().max()) <= 1e-3
            assert float((got[0].float() - want[0].transpose(0, 1).float()).abs().max()) <= 2e-2


def test_python_refusals(attn):
    q = normal((2, 4, 64), 1).cuda()
    c = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    t, cu, n = ints([[0], [1]]).cuda(), ints([0, 1, 2]).cuda(), ints([3, 4]).cuda()
    c8 = c.to(torch.float8_e4m3fn)
    s8 = torch.zeros(3, 2, 16, dtype=torch.uint8, device="cuda")
    good = (q, c, c, t, cu, n)
    attn.attn_paged(*good)
    ok(attn)

    def bad(exc, *args, **kw):
        with pytest.raises(exc):
            attn.attn_paged(*args, **kw)
    bad(TypeError, q.float(), c, c, t, cu, n)
    bad(ValueError, q.transpose(1, 2), c, c, t, cu, n)
    bad(ValueError, q, c, c[:2], t, cu, n)
    bad(ValueError, q, c, c, t[:1], cu, n)
    bad(ValueError, q, c, c, t, cu[:2], n)
    bad(TypeError, q, c, c, t.long(), cu, n)
    bad(ValueError, q, c, c, t, cu, n, k_scale=s8, v_scale=s8)
    bad(TypeError, q, c8, c8, t, cu, n)
    bad(ValueError, q, c.transpose(1, 2), c.transpose(1, 2), t, cu, n)
    bad(ValueError, *good, o=torch.empty(2, 4, 128, dtype=torch.bfloat16, device="cuda"))
    bad(attn.AttnError, *good, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    bad(attn.AttnError, *good, scale=-1.0)
    f = attn.rope_inv_freq(64)[0]
    with pytest.raises(ValueError):
        attn.attn_cache_write(c[:2, :, 0], c[:2, :, 0], c, c, t, cu, n, q=q)           # q without inv_freq
    with pytest.raises(ValueError):
        attn.attn_rope(q, positions=n[:1], inv_freq=f)
    with pytest.raises(TypeError):
        attn.attn_rope(q, positions=n, inv_freq=f.float())
    with pytest.raises(ValueError):
        attn.attn_cache_read(c, c, t, n)                                               # no N
