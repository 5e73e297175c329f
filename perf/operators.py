"""The serving operators as a user calls them: rotary positions, the paged cache's write
and read-back, and attention of new tokens over the paged cache.

Every case is a dict of plain values with an ``op``:

- ``rope``: rotary positions of q and k (``grad``: the transposed rotation of their
  gradients), dense [B, H, N, d] or packed [T, H, d];
- ``write``: one step's new tokens go into a bf16 paged cache, K and Q rotated on the way;
- ``store``: new tokens are quantised to an e4m3 paged cache and read back as the bf16
  values that the codes stand for;
- ``read``: a paged cache is gathered into the dense layout;
- ``paged``: attention of packed new tokens over a paged cache.

A sequence's lengths follow from the case alone (``lengths``); its pages are a random
permutation of the pool.  The e4m3 cache keeps a power-of-two scale per token and KV head,
2^(byte - 127): the smallest one that brings the row's largest finite magnitude to 448.
"""
import math
import random

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of 8 requests before a cache is written: latency
        dict(name="rope_step_8", op="rope", layout="packed", B=1, N=8, Hq=32, Hkv=8, d=128, rot=128, interleaved=False,
             dtype="bf16", grad=False, mscale=1.0, far=32768),
        # a training batch of grouped heads at 8K, whole head rotated
        dict(name="rope_train_gqa_8k", op="rope", layout="dense", B=4, N=8192, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, dtype="bf16", grad=False, mscale=1.0, far=8192),
        # gradients in fp32 (as a ring sums them), half of the head interleaved, odd length, scaled for long contexts
        dict(name="rope_grad_odd_f32", op="rope", layout="dense", B=16, N=1001, Hq=16, Hkv=16, d=64, rot=32,
             interleaved=True, dtype="f32", grad=True, mscale=1.1386, far=131072),
        # one decoding step of 64 requests: rotate Q and K, put K and V into the cache
        dict(name="write_step_64", op="write", B=64, new=1, ctx=8192, Hq=32, Hkv=8, d=128, page=64, rot=128,
             interleaved=False),
        # prompts' chunks of plain multi-head attention, ragged, part of the head interleaved
        dict(name="write_chunk_mha_d64", op="write", B=6, new=2048, ctx=4096, Hq=16, Hkv=16, d=64, page=32, rot=32,
             interleaved=True),
        # prompts' chunks quantised to 8 bits and read back
        dict(name="store_chunk_e4m3", op="store", B=5, new=4096, ctx=4096, Hkv=8, d=128, page=16),
        # a bf16 cache gathered for a dense pass
        dict(name="read_bf16_16k", op="read", B=8, ctx=16384, Hkv=8, d=128, page=64, kv="bf16"),
        # one request, a short context: latency
        dict(name="decode_one_1k", op="paged", B=1, new=1, one=0, ctx=1000, Hq=32, Hkv=8, d=128, page=64, kv="bf16",
             window=-1),
        # a batch of requests in the middle of long contexts: the cache's bandwidth
        dict(name="decode_16_32k", op="paged", B=16, new=1, one=0, ctx=32768, Hq=32, Hkv=8, d=128, page=64, kv="bf16",
             window=-1),
        # many requests over an 8-bit cache of small pages
        dict(name="decode_64_8k_e4m3", op="paged", B=64, new=1, one=0, ctx=8192, Hq=32, Hkv=8, d=128, page=16,
             kv="e4m3", window=-1),
        # a long prompt's last chunk over what is already cached: the tensor cores
        dict(name="chunk_4k_on_28k", op="paged", B=1, new=4096, one=0, ctx=32768, Hq=32, Hkv=8, d=128, page=128,
             kv="bf16", window=-1),
        # chunks and single tokens in one batch, 5 query heads to a KV head, a sliding window, 8 bits
        dict(name="mixed_window_e4m3_d64", op="paged", B=24, new=777, one=16, ctx=6000, Hq=20, Hkv=4, d=64, page=32,
             kv="e4m3", window=1023),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "write", "store", "read", "paged", "paged", "paged", "paged"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    if op == "rope":
        dense = rng.random() < 0.7
        B, N = (rng.randint(1, 8), _log(rng, 17, 8192)) if dense else (1, _log(rng, 1, 16384))
        Hq = Hkv * rng.choice([1, 2, 4])
        while B * N * (Hq + Hkv) * d > 4 * 8192 * 40 * 128 // 2:
            N = max(1, N // 2)
        return dict(op=op, layout="dense" if dense else "packed", B=B, N=N, Hq=Hq, Hkv=Hkv, d=d,
                    rot=rng.choice([16, 32, d // 2, d]), interleaved=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), grad=rng.random() < 0.4,
                    mscale=rng.choice([1.0, 1.1386]), far=rng.choice([8192, 131072, 1000000]))
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "write":
        B, new = rng.choice([(rng.randint(1, 128), 1), (rng.randint(1, 8), _log(rng, 2, 2048))])
        return dict(op=op, B=B, new=new, ctx=max(new, _log(rng, 100, 8192)), Hq=Hkv * rng.choice([1, 3, 4]), Hkv=Hkv, d=d,
                    page=page, rot=rng.choice([16, 32, d // 2, d]), interleaved=rng.random() < 0.5)
    if op == "store":
        new = _log(rng, 1, 4096)
        return dict(op=op, B=rng.randint(1, 8), new=new, ctx=new + rng.choice([0, rng.randint(1, 2000)]), Hkv=Hkv, d=d, page=page)
    if op == "read":
        return dict(op=op, B=rng.randint(1, 8), ctx=_log(rng, 1, 16384), Hkv=min(Hkv, 8), d=d, page=page,
                    kv=rng.choice(["bf16", "e4m3"]))
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 8])
    kind = rng.choice(["decode", "decode", "few", "chunk", "mixed"])
    B, one = rng.randint(1, 64), 0
    if kind == "decode":
        new, ctx = 1, _log(rng, 50, 32768)
    elif kind == "few":
        new = rng.randint(2, 12)
        ctx = max(new, _log(rng, 50, 16384))
    elif kind == "chunk":
        B, new = rng.randint(1, 3), _log(rng, 13, 2048)
        ctx = max(new, _log(rng, 50, 16384))
    else:
        B, new = rng.randint(2, 24), _log(rng, 13, 800)
        one = rng.randint(1, B - 1)
        ctx = max(new, _log(rng, 50, 8192))
    while B > 1 and B * ctx * Hkv > 16 * 32768 * 8:
        B = (B + 1) // 2
        one = min(one, B - 1)
    return dict(op="paged", B=B, new=new, one=one, ctx=ctx, Hq=Hkv * G, Hkv=Hkv, d=d, page=page,
                kv=rng.choice(["bf16", "e4m3"]), window=rng.choice([-1, -1, -1, rng.randint(0, ctx)]))


def lengths(case):
    """Per sequence (new tokens, tokens in the cache with them), ragged: the first sequence is the
    longest, the last ``one`` have a single new token."""
    B, new, one = case["B"], case.get("new", 0), case.get("one", 0)
    rng = random.Random(B * 1000003 + case["ctx"] * 101 + new)
    out = []
    for b in range(B):
        n = new if b == 0 or new <= 1 else rng.randint(max(1, new // 2), new)
        if b >= B - one:
            n = 1
        length = case["ctx"] if b == 0 else rng.randint(max(n, (case["ctx"] + 1) // 2), case["ctx"])
        out.append((n, max(n, length)))
    return out


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype):
    x = torch.empty(shape, device="cuda", dtype=dtype)
    return x.normal_(generator=gen)


def _inv_freq(rot, base=10000.0):
    i = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda")
    return base ** (-i / rot)


def _quantise(x):
    """e4m3 codes and power-of-two scale bytes of bf16 rows [..., d]."""
    f = x.float()
    amax = f.abs().amax(dim=-1)
    m, e = torch.frexp(amax)                              # amax = m 2^e, m in [1/2, 1)
    k = torch.where(m <= 0.875, e - 9, e - 8)             # amax 2^-k <= 448
    k = torch.where(amax > 0, k, torch.full_like(k, -127)).clamp(-127, 120)
    codes = torch.ldexp(f, -k.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes, (k + 127).to(torch.uint8)


def _pool(case, gen, lens, fill):
    """A page pool with room to spare, and the table of a random choice of its pages."""
    page, Hkv, d = case["page"], case["Hkv"], case["d"]
    need = [-(-L // page) for L in lens]
    total, width = sum(need), max(1, max(need))
    pages = total + max(2, total // 8)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((case["B"], width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (pages, Hkv, page, d)
    pool = {"table": table}
    e4m3 = case.get("kv", "bf16") == "e4m3"
    for name in ("k", "v"):
        if not fill:
            pool[name] = torch.zeros(shape, device="cuda", dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16)
            pool[name + "_scale"] = torch.zeros(shape[:3], device="cuda", dtype=torch.uint8) if e4m3 else None
        elif e4m3:
            codes = torch.empty(shape, device="cuda", dtype=torch.float8_e4m3fn)
            scales = torch.empty(shape[:3], device="cuda", dtype=torch.uint8)
            step = max(1, (1 << 26) // (Hkv * page * d))
            for p in range(0, pages, step):
                c, s = _quantise(_normal(gen, (min(step, pages - p), Hkv, page, d), torch.bfloat16))
                codes[p:p + step], scales[p:p + step] = c, s
            pool[name], pool[name + "_scale"] = codes, scales
        else:
            pool[name], pool[name + "_scale"] = _normal(gen, shape, torch.bfloat16), None
    return pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, d = case["op"], case["d"]
    st = dict(case=case)
    if op == "rope":
        B, N, Hq, Hkv = case["B"], case["N"], case["Hq"], case["Hkv"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        shape = (lambda H: (B, H, N, d)) if case["layout"] == "dense" else (lambda H: (N, H, d))
        st["q"], st["k"] = _normal(gen, shape(Hq), dt), _normal(gen, shape(Hkv), dt)
        if case["layout"] == "dense":
            first = torch.randint(0, max(1, case["far"] - N + 1), (B, 1), generator=gen, device="cuda")
            st["positions"] = (first + torch.arange(N, device="cuda")).to(torch.int32)
        else:
            st["positions"] = torch.randint(0, case["far"], (N,), generator=gen, device="cuda").to(torch.int32)
        st["inv_freq"] = _inv_freq(case["rot"])
        return st
    pairs = lengths(case)
    st["new"], st["len"] = [n for n, _ in pairs], [L for _, L in pairs]
    st.update(_pool(case, gen, st["len"], fill=op in ("read", "paged")) if op != "store"
              else _pool(dict(case, kv="e4m3"), gen, st["len"], fill=False))
    st["kv_len"] = torch.tensor(st["len"], dtype=torch.int32, device="cuda")
    st["cu_q"] = torch.tensor([0] + list(np.cumsum(st["new"])), dtype=torch.int32, device="cuda")
    T = sum(st["new"])
    if op == "write":
        # one fused projection's output, q, k and v side by side: strided views
        Hq, Hkv = case["Hq"], case["Hkv"]
        qkv = _normal(gen, (T, Hq + 2 * Hkv, d), torch.bfloat16)
        st["q"], st["knew"], st["vnew"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        st["inv_freq"] = _inv_freq(case["rot"])
        st["q_out"] = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda")
    elif op == "store":
        kv = _normal(gen, (T, 2 * case["Hkv"], d), torch.bfloat16)
        st["knew"], st["vnew"] = kv[:, :case["Hkv"]], kv[:, case["Hkv"]:]
    elif op == "paged":
        st["q"] = _normal(gen, (T, case["Hq"], d), torch.bfloat16)
        if own:
            import io_aware_exact_26_b200 as attn
            size = attn.attn_paged_workspace_size(T, case["B"], case["Hq"], case["Hkv"], d)
            st["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    if op in ("store", "read"):
        shape = (case["B"], case["Hkv"], case["ctx"], d)
        st["k_out"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        st["v_out"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import io_aware_exact_26_b200 as attn
    case = st["case"]
    op = case["op"]
    if op == "rope":
        call = attn.attn_rope_bwd if case["grad"] else attn.attn_rope
        q, k = call(st["q"], st["k"], positions=st["positions"], inv_freq=st["inv_freq"],
                    interleaved=case["interleaved"], mscale=case["mscale"])
        return {"q": q, "k": k}
    where = (st["k"], st["v"], st["table"])
    if op == "write":
        q = attn.attn_cache_write(st["knew"], st["vnew"], *where, st["cu_q"], st["kv_len"], inv_freq=st["inv_freq"],
                                  interleaved=case["interleaved"], q=st["q"], q_out=st["q_out"])
        return {"q": q, "k": st["k"], "v": st["v"]}
    scales = dict(k_scale=st["k_scale"], v_scale=st["v_scale"])
    if op == "store":
        attn.attn_cache_write(st["knew"], st["vnew"], *where, st["cu_q"], st["kv_len"], **scales)
    if op in ("store", "read"):
        k, v = attn.attn_cache_read(*where, st["kv_len"], **scales, k_out=st["k_out"], v_out=st["v_out"])
        return {"k": k, "v": v}
    o, lse = attn.attn_paged(st["q"], *where, st["cu_q"], st["kv_len"], **scales, causal=True,
                             window_left=case["window"], workspace=st["workspace"])
    return {"o": o, "lse": lse}


def _rotate(x, angle, rot, interleaved, mscale, back=False):
    """x [..., d] fp32, angle [..., rot/2] fp64 broadcast over heads: m R x, or m R^T x."""
    cos, sin = (angle.cos() * mscale).float(), (angle.sin() * mscale).float()
    if back:
        sin = -sin
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = x.clone()
    ya, yb = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = ya, yb
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ya, yb
    return y


def _places(st):
    """Of every new token: its sequence, its position, its page and its row there."""
    page, dev = st["case"]["page"], st["table"].device
    T = st["knew"].shape[0]
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(st["cu_q"].long(), t, right=True) - 1
    p = st["kv_len"].long()[b] - st["cu_q"].long()[b + 1] + t
    return b, p, st["table"].long()[b, p // page], p % page


def _gathered(st, name, b, L):
    """Positions [0, L) of sequence b as fp32 [Hkv, L, d]."""
    page = st["case"]["page"]
    ids = st["table"][b, :-(-L // page)].long()
    x = st[name][ids].float()
    if st[name + "_scale"] is not None:
        x = torch.ldexp(x, st[name + "_scale"][ids].to(torch.int32).unsqueeze(-1) - 127)
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :L]


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "rope":
        angle = st["positions"].double().unsqueeze(-1) * st["inv_freq"]
        angle = angle.unsqueeze(1)                       # [B, 1, N, rot/2] or [T, 1, rot/2]
        return {n: _rotate(st[n].float(), angle, case["rot"], case["interleaved"], case["mscale"], case["grad"]).to(st[n].dtype)
                for n in ("q", "k")}
    if op in ("write", "store"):
        _, pos, ids, row = _places(st)
        if op == "write":
            angle = (pos.double().unsqueeze(-1) * st["inv_freq"]).unsqueeze(1)
            turn = lambda x: _rotate(x.float(), angle, case["rot"], case["interleaved"], 1.0).to(torch.bfloat16)  # noqa: E731
            st["q_out"].copy_(turn(st["q"]))
            st["k"][ids, :, row] = turn(st["knew"])
            st["v"][ids, :, row] = st["vnew"]
            return {"q": st["q_out"], "k": st["k"], "v": st["v"]}
        for name in ("k", "v"):
            codes, scales = _quantise(st[name + "new"])
            st[name].view(torch.uint8)[ids, :, row] = codes.view(torch.uint8)
            st[name + "_scale"][ids, :, row] = scales
    if op in ("store", "read"):
        for b, L in enumerate(st["len"]):
            for name in ("k", "v"):
                st[name + "_out"][b, :, :L] = _gathered(st, name, b, L).to(torch.bfloat16)
        return {"k": st["k_out"], "v": st["v_out"]}
    T, Hq, d = st["q"].shape
    G = Hq // case["Hkv"]
    o = torch.empty_like(st["q"])
    lse = torch.empty((T, Hq), dtype=torch.float32, device=o.device)
    t0 = 0
    for b, (n, L) in enumerate(zip(st["new"], st["len"])):
        k, v = _gathered(st, "k", b, L), _gathered(st, "v", b, L)
        step = max(1, (1 << 28) // (Hq * L))
        key = torch.arange(L, device=o.device)
        for i in range(0, n, step):
            m = min(step, n - i)
            q = st["q"][t0 + i:t0 + i + m].float().reshape(m, -1, G, d).permute(1, 0, 2, 3).reshape(-1, m * G, d)
            s = torch.matmul(q, k.transpose(1, 2)) * d ** -0.5
            pos = (L - n + i + torch.arange(m, device=o.device)).repeat_interleave(G).unsqueeze(1)
            hide = key > pos
            if case["window"] >= 0:
                hide = hide | (key < pos - case["window"])
            s.masked_fill_(hide, float("-inf"))
            top = s.amax(dim=-1, keepdim=True)
            s = s.sub_(top).exp_()
            total = s.sum(dim=-1, keepdim=True)
            out = torch.matmul(s, v) / total
            o[t0 + i:t0 + i + m] = out.reshape(-1, m, G, d).permute(1, 0, 2, 3).reshape(m, Hq, d).to(o.dtype)
            lse[t0 + i:t0 + i + m] = (top + total.log()).reshape(-1, m, G).permute(1, 0, 2).reshape(m, Hq)
        t0 += n
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    if op == "rope":
        el = case["B"] * case["N"] * (case["Hq"] + Hkv) * d
        return {"bytes": 2 * el * (2 if case["dtype"] == "bf16" else 4) + case["B"] * case["N"] * 4 + case["rot"] * 4,
                "flops": 3 * el * case["rot"] // d}
    pairs = lengths(case)
    T, total = sum(n for n, _ in pairs), sum(L for _, L in pairs)
    if op == "write":
        rows = T * (case["Hq"] + 2 * Hkv)
        return {"bytes": 2 * rows * d * 2 + T * 4, "flops": 3 * T * (case["Hq"] + Hkv) * case["rot"]}
    cached = 2 * total * Hkv * (d * 2 if case.get("kv") == "bf16" else d + 1)
    if op == "store":
        return {"bytes": 2 * T * Hkv * (d * 2 + d + 1) + cached + 2 * total * Hkv * d * 2, "flops": 4 * T * Hkv * d}
    if op == "read":
        return {"bytes": cached + 2 * total * Hkv * d * 2, "flops": 2 * total * Hkv * d}
    keys = seen = 0
    for n, L in pairs:
        w = case["window"] if case["window"] >= 0 else L
        seen += sum(min(p, w) + 1 for p in range(L - n, L))
        keys += L - max(0, L - n - w)
    es = d * 2 if case["kv"] == "bf16" else d + 1
    return {"bytes": 2 * keys * Hkv * es + T * case["Hq"] * (d * 4 + 4), "flops": 4 * case["Hq"] * d * seen}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "rope":
        return {n: _turned(st[n], st["positions"], st["inv_freq"], case, case["mscale"], -1 if case["grad"] else 1)
                for n in ("q", "k")}
    if op in ("write", "store"):
        at = 0
        cache = {n: st[n].double() for n in ("k", "v")}
        q = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda") if op == "write" else None
        for b, (n, L) in enumerate(lengths(case)):
            pos = torch.arange(L - n, L, device="cuda")
            ids, row = st["table"][b].long()[pos // case["page"]], pos % case["page"]
            part = slice(at, at + n)
            new = {"k": st["knew"][part], "v": st["vnew"][part]}
            if op == "write":
                new["k"] = _turned(new["k"], pos, st["inv_freq"], case, 1.0, 1)
                q[part] = _turned(st["q"][part], pos, st["inv_freq"], case, 1.0, 1)
            for name in ("k", "v"):
                x = new[name].double()
                cache[name][ids, :, row] = x if op == "write" else _eight_bits(x)
            at += n
        if op == "write":
            return {"q": q, "k": cache["k"], "v": cache["v"]}
    if op == "read":
        cache = {}
        for name in ("k", "v"):
            cache[name] = st[name].double()
            if st[name + "_scale"] is not None:
                cache[name] *= torch.exp2(st[name + "_scale"].double() - 127).unsqueeze(-1)
    if op in ("store", "read"):
        out = {n: torch.zeros((case["B"], case["Hkv"], case["ctx"], d), dtype=torch.float64, device="cuda") for n in ("k", "v")}
        for b, (_, L) in enumerate(lengths(case)):
            pos = torch.arange(L, device="cuda")
            ids, row = st["table"][b].long()[pos // case["page"]], pos % case["page"]
            for name in ("k", "v"):
                out[name][b, :, :L] = cache[name][ids, :, row].transpose(0, 1)
        return out
    if work(case)["flops"] > 2e14:
        return None
    G, scale = case["Hq"] // case["Hkv"], 1.0 / math.sqrt(d)
    o = torch.zeros((sum(st["new"]), case["Hq"], d), dtype=torch.float64, device="cuda")
    lse = torch.zeros(o.shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, L) in enumerate(lengths(case)):
        pos = torch.arange(L, device="cuda")
        ids, row = st["table"][b].long()[pos // case["page"]], pos % case["page"]
        for g in range(case["Hkv"]):
            k, v = (_head(st, name, ids, row, g) for name in ("k", "v"))
            for h in range(g * G, g * G + G):
                for i in range(0, n, 1024):
                    who = torch.arange(i, min(n, i + 1024), device="cuda")
                    at_pos = (L - n + who).unsqueeze(1)
                    seen = pos <= at_pos
                    if case["window"] >= 0:
                        seen &= pos >= at_pos - case["window"]
                    s = torch.where(seen, st["q"][at + who, h].double() @ k.T * scale, -math.inf)
                    o[at + who, h] = torch.softmax(s, dim=-1) @ v
                    lse[at + who, h] = torch.logsumexp(s, dim=-1)
        at += n
    return {"o": o, "lse": lse}


def _head(st, name, ids, row, g):
    x = st[name][ids, g, row].double() if st[name].dtype == torch.bfloat16 else st[name].view(torch.uint8)[ids, g, row].view(
        torch.float8_e4m3fn).double()
    scale = st[name + "_scale"]
    return x if scale is None else x * torch.exp2(scale[ids, g, row].double() - 127).unsqueeze(-1)


def _turned(x, positions, inv_freq, case, mscale, sign):
    """The complex form: each pair is a number turned by e^(i sign angle)."""
    rot = case["rot"]
    turn = torch.polar(torch.full((), mscale, dtype=torch.float64, device="cuda"),
                       sign * positions.double().unsqueeze(-1) * inv_freq).unsqueeze(1)
    y = x.double()
    if case["interleaved"]:
        z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2).contiguous()) * turn
        part = torch.view_as_real(z).reshape(*y.shape[:-1], rot)
    else:
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
        part = torch.cat([z.real, z.imag], dim=-1)
    return torch.cat([part, y[..., rot:]], dim=-1)


def _eight_bits(x):
    """Rows rounded to 3 mantissa bits of e4m3 under their power-of-two scale, ties to even."""
    amax = x.abs().amax(dim=-1, keepdim=True)
    e = torch.where(amax > 0, torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448.0)), torch.full_like(amax, -127.0))
    unit = torch.exp2(e)
    y = x / unit
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step * unit
