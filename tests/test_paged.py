"""The serving operators without a GPU: refusals at the C entry points, the binding's own
checks, and the frequencies of the rotary pairs."""
import ctypes
import math
import os
import re

import pytest
import torch

import __graft_entry__
import io_aware_exact_26_b200 as attn
from io_aware_exact_26_b200 import binding, paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, ODD, NULL = 0x10000, 0x10008, None      # never dereferenced: every call here is refused


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return binding.lib()


def test_every_serving_symbol_is_exported(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "attn_paged.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(attn_[a-z0-9_]+)\s*\(", text)))
    assert names == ["attn_cache_read", "attn_cache_write", "attn_paged", "attn_paged_workspace_size", "attn_rope"]
    checks = binding.load(binding.checks_library_path)
    for n in names:
        assert hasattr(L, n) and hasattr(checks, n), n


def test_bad_page_status_has_its_text(L):
    texts = {binding.attn_status_string(c) for c in range(-10, 1)}
    assert len(texts) == 11 and "unknown status" not in texts


def cache(**kw):
    c = dict(k=FAKE, v=FAKE, k_scale=NULL, v_scale=NULL, page_stride=4 * 64 * 128, num_pages=10, page_size=64, Hkv=4,
             d=128, dtype=0)
    c.update(kw)
    return paged._Cache(*c.values())


def batch(**kw):
    b = dict(cu_q=FAKE, kv_len=FAKE, block_table=FAKE, B=2, T=9, max_pages=5)
    b.update(kw)
    return paged._Batch(*b.values())


def strides(batch=0, head=128, token=1024):
    return paged._Strides(batch, head, token)


def rope(**kw):
    r = dict(inv_freq=FAKE, rot=128, interleaved=0, mscale=1.0)
    r.update(kw)
    return paged._Rope(*r.values())


CACHE_REFUSALS = [
    (dict(d=96), -2), (dict(dtype=1), -1), (dict(dtype=7), -1), (dict(page_size=8), -1), (dict(page_size=48), -1),
    (dict(page_size=512), -1), (dict(num_pages=0), -1), (dict(Hkv=0), -1), (dict(page_stride=4 * 64 * 128 - 8), -1),
    (dict(page_stride=4 * 64 * 128 + 4), -1), (dict(k=NULL), -1), (dict(v=NULL), -1), (dict(dtype=2), -1),
    (dict(dtype=2, k_scale=FAKE), -1), (dict(k=ODD), -3), (dict(v=ODD), -3),
    (dict(dtype=2, k_scale=FAKE, v_scale=ODD), -3),
]
BATCH_REFUSALS = [(dict(B=0), -1), (dict(max_pages=0), -1), (dict(kv_len=NULL), -1), (dict(block_table=NULL), -1),
                  (dict(kv_len=FAKE + 2), -3)]
PACKED_REFUSALS = [(dict(cu_q=NULL), -1), (dict(T=-1), -1), (dict(cu_q=FAKE + 2), -3)]


def call_paged(L, c=None, b=None, q=FAKE, st=None, o=FAKE, lse=FAKE, Hq=8, scale=0.1, causal=1, window=-1, ws=NULL, wsb=0):
    return L.attn_paged(q, st or strides(), c or cache(), b or batch(), o, lse, Hq, scale, causal, window, ws, wsb, NULL)


def call_write(L, c=None, b=None, k=FAKE, ks=None, v=FAKE, r=None, q=NULL, q_out=NULL, Hq=0, qs=None):
    return L.attn_cache_write(c or cache(), b or batch(), k, ks or strides(), v, strides(), r, q, qs or strides(), q_out,
                              strides(), Hq, NULL)


def call_read(L, c=None, b=None, k=FAKE, v=FAKE, N=100):
    return L.attn_cache_read(c or cache(), b or batch(), k, v, N, NULL)


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS)
def test_cache_descriptor_refusals(L, kw, code):
    assert call_paged(L, c=cache(**kw)) == code
    assert call_write(L, c=cache(**kw)) == code
    assert call_read(L, c=cache(**kw)) == code


@pytest.mark.parametrize("kw,code", BATCH_REFUSALS + PACKED_REFUSALS)
def test_batch_descriptor_refusals(L, kw, code):
    assert call_paged(L, b=batch(**kw)) == code
    assert call_write(L, b=batch(**kw)) == code
    if (kw, code) in BATCH_REFUSALS:
        assert call_read(L, b=batch(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=NULL), -1), (dict(o=NULL), -1), (dict(lse=NULL), -1), (dict(Hq=0), -1), (dict(Hq=6), -1),
    (dict(Hq=4 * 129), -1), (dict(scale=-1.0), -1), (dict(scale=math.nan), -1), (dict(scale=math.inf), -1),
    (dict(causal=2), -1), (dict(q=ODD), -3), (dict(o=ODD), -3), (dict(lse=ODD), -3), (dict(ws=ODD, wsb=1 << 30), -3),
    (dict(st=strides(token=1020)), -1), (dict(st=strides(head=-128)), -1)])
def test_paged_refusals(L, kw, code):
    assert call_paged(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=NULL), -1), (dict(v=NULL), -1), (dict(k=ODD), -3), (dict(v=ODD), -3), (dict(ks=strides(token=4)), -1),
    (dict(r=rope(rot=24)), -1), (dict(r=rope(rot=0)), -1), (dict(r=rope(rot=144)), -1), (dict(r=rope(inv_freq=NULL)), -1),
    (dict(r=rope(inv_freq=ODD)), -3), (dict(r=rope(mscale=math.inf)), -1), (dict(r=rope(interleaved=2)), -1),
    (dict(q=FAKE, q_out=FAKE, Hq=8), -1), (dict(r=rope(), q=FAKE, q_out=NULL, Hq=8), -1),
    (dict(r=rope(), q=FAKE, q_out=FAKE, Hq=0), -1), (dict(r=rope(), q=ODD, q_out=FAKE, Hq=8), -3)])
def test_write_refusals(L, kw, code):
    assert call_write(L, **kw) == code


@pytest.mark.parametrize("kw,code", [(dict(k=NULL), -1), (dict(v=NULL), -1), (dict(N=-1), -1), (dict(k=ODD), -3),
                                     (dict(v=ODD), -3), (dict(b=batch(B=20000)), -1)])
def test_read_refusals(L, kw, code):
    assert call_read(L, **kw) == code


def call_rope(L, q=FAKE, q_out=FAKE, Hq=4, k=NULL, k_out=NULL, Hkv=0, dtype=0, B=1, N=5, d=128, pos=FAKE, ps=0, r=None,
              inv=0, st=None):
    s = st or strides(5 * 4 * 128, 5 * 128, 128)
    return L.attn_rope(q, s, q_out, s, Hq, k, s, k_out, s, Hkv, dtype, B, N, d, pos, ps, r or rope(), inv, NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), -2), (dict(dtype=2), -1), (dict(q=NULL), -1), (dict(q_out=NULL), -1), (dict(pos=NULL), -1),
    (dict(Hq=0), -1), (dict(B=-1), -1), (dict(N=-1), -1), (dict(inv=2), -1), (dict(ps=-1), -1), (dict(q=ODD), -3),
    (dict(q_out=ODD), -3), (dict(pos=FAKE + 2), -3), (dict(k=FAKE, Hkv=1), -1), (dict(k=FAKE, k_out=FAKE), -1),
    (dict(k=FAKE, k_out=ODD, Hkv=1), -3), (dict(r=rope(rot=20)), -1), (dict(d=64, r=rope(rot=128)), -1),
    (dict(st=strides(0, 0, 4)), -1), (dict(B=1 << 16, N=1 << 16), -1)])
def test_rope_refusals(L, kw, code):
    assert call_rope(L, **kw) == code


def test_nothing_to_do_is_not_an_error(L):
    assert call_paged(L, b=batch(T=0), q=NULL, o=NULL, lse=NULL) == 0
    assert call_write(L, b=batch(T=0), k=NULL, v=NULL) == 0
    assert call_read(L, N=0, k=NULL, v=NULL) == 0
    assert call_rope(L, N=0, q=NULL, q_out=NULL, pos=NULL) == 0
    assert L.attn_paged_workspace_size(0, 1, 8, 2, 128) == 0


def test_workspace_size_refuses_what_the_call_refuses(L):
    for bad in [(4, 1, 8, 2, 96), (4, 0, 8, 2, 128), (4, 1, 9, 2, 128), (4, 1, 258, 1, 64), (-1, 1, 8, 2, 64)]:
        assert L.attn_paged_workspace_size(*bad) == 0


def test_binding_refuses_tensors_that_are_not_on_a_gpu(L):
    c = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    t, n = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_paged(torch.zeros(1, 2, 64, dtype=torch.bfloat16), c, c, t, torch.zeros(2, dtype=torch.int32), n)
    with pytest.raises(TypeError):
        attn.attn_rope(torch.zeros(1, 2, 64, dtype=torch.float16), positions=n, inv_freq=n)
    with pytest.raises(ValueError):
        attn.attn_rope(torch.zeros(1, 2, 64), positions=n, inv_freq=n)


# ------------------------------------------------------------------ frequencies
def test_inv_freq_plain_and_scaled():
    rot, base, s = 64, 10000.0, 8.0
    f, m = attn.rope_inv_freq(rot, base, device="cpu")
    want = torch.tensor([base ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    assert m == 1.0 and f.dtype == torch.float64 and torch.allclose(f, want, rtol=1e-14)
    g, m = attn.rope_inv_freq(rot, base, scaling="linear", factor=s, device="cpu")
    assert m == 1.0 and torch.allclose(g, want / s, rtol=1e-14)
    g, m = attn.rope_inv_freq(rot, base, scaling="ntk", factor=s, device="cpu")
    assert m == 1.0 and float(g[0]) == 1.0 and math.isclose(float(g[-1]), float(want[-1]) / s, rel_tol=1e-12)


def test_inv_freq_yarn_keeps_fast_pairs_and_slows_slow_ones():
    rot, base, s, n = 128, 10000.0, 4.0, 4096
    f, _ = attn.rope_inv_freq(rot, base, device="cpu")
    g, m = attn.rope_inv_freq(rot, base, scaling="yarn", factor=s, original=n, device="cpu")
    turns = n * f / (2 * math.pi)
    ratio = g / f
    assert math.isclose(m, 0.1 * math.log(s) + 1.0)
    # the ramp runs between whole pair indices, so a pair just inside an end may be off by one index
    assert torch.allclose(ratio[turns > 32 * base ** (2 / rot)], torch.ones((), dtype=torch.float64), rtol=1e-12)
    assert torch.allclose(ratio[turns < 1 / base ** (2 / rot)], torch.full((), 1 / s, dtype=torch.float64), rtol=1e-12)
    assert bool((ratio[1:] <= ratio[:-1] + 1e-12).all())


@pytest.mark.parametrize("kw", [dict(rot=8), dict(rot=40), dict(rot=64, base=1.0), dict(rot=64, factor=0.5),
                                dict(rot=64, scaling="other"), dict(rot=64, scaling="yarn", factor=2.0),
                                dict(rot=64, scaling="yarn", factor=2.0, original=4096, beta_fast=1.0, beta_slow=2.0)])
def test_inv_freq_refusals(kw):
    with pytest.raises(ValueError):
        attn.rope_inv_freq(device="cpu", **kw)


# ------------------------------------------------------------------ positions of ring shards
@pytest.mark.parametrize("layout", ["contiguous", "zigzag"])
@pytest.mark.parametrize("world", [1, 2, 4])
def test_shard_positions_rotate_a_shard_like_the_whole_sequence(layout, world):
    from io_aware_exact_26_b200 import ring
    from tests import paged_reference as ref
    N, d = 48, 64
    x = torch.randn(N, 2, d, generator=torch.Generator().manual_seed(1))
    f = attn.rope_inv_freq(d, device="cpu")[0]
    whole = ref.rotate(x, torch.arange(N), f, False)
    seen = []
    for rank in range(world):
        pos = ring.shard_positions(rank, world, N, layout)
        assert pos.dtype == torch.int32 and pos.shape == (N // world,)
        assert torch.equal(ref.rotate(x[pos.long()], pos, f, False), whole[pos.long()])
        n = N // (world * len(ring.shard_chunks(rank, world, layout)))
        assert pos[::n].tolist() == [c * n for c in ring.shard_chunks(rank, world, layout)]
        seen += pos.tolist()
    assert sorted(seen) == list(range(N))
    with pytest.raises(ValueError):
        ring.shard_positions(0, 5, N, layout)
