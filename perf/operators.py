"""The rotary-position, rotating-append and chunk-attention operators, as cases that can be timed.

Four operators of the paged cache's prefill path, each in its plain form (elementary torch
operations) and, with ``own`` true, through the library's entry points:

- ``table``   : cos / sin of every position, scaled for long contexts (``kvq_rope_table``);
- ``rope``    : the rotation of query (or key) rows by their positions, and its inverse, which is
  also its backward pass (``kvq_rope``);
- ``append``  : keys (rotated on the way) and values into a paged cache, INT2 or BF16
  (``kvq_append_rope``, ``kvq_bf16_append_rope``);
- ``prefill`` : causal attention of each sequence's new tokens over its paged cache, INT2 or BF16
  (``kvq_prefill``, ``kvq_bf16_prefill``).

Head dimension 128 and 16-token pages, the cache's own; the page records' byte layouts are those
of include/kvq.h.  Everything is made from the seed alone.
"""
import math

import numpy as np
import torch

own = False

D, PAGE = 128, 16
INT2_REC, BF16_REC = 1152, 8192
CLIP_K, CLIP_V = 0.96, 0.92


# ---- cases --------------------------------------------------------------------------------------

def listed():
    """Twelve cases.  32 query heads over 8 KV heads, batch 16, 32K contexts and the 64-sequence
    ragged batch are this library's benchmark shapes; the others are generic."""
    return [
        # one decode step's queries, 16 sequences: a launch and little else
        dict(name="rope_step_16", op="rope", n=16, heads=32, rot=128, style="half",
             inverse=False, fused_qkv=False, table_len=32768),
        # a long prompt's queries inside the fused projection's output, half of each head rotated
        dict(name="rope_chunk_8191", op="rope", n=8191, heads=32, rot=64, style="interleaved",
             inverse=False, fused_qkv=True, table_len=32768),
        # the table of a short-context model
        dict(name="table_8k", op="table", table_len=8192, rot=128, kind="none", base=1e4,
             factor=1.0, orig_len=8192),
        # the table of a model stretched from 32K to 128K
        dict(name="table_128k_yarn", op="table", table_len=131072, rot=128, kind="yarn", base=1e6,
             factor=4.0, orig_len=32768),
        # one decode step's new tokens, 16 sequences
        dict(name="append_int2_step_16", op="append", cache="int2", batch=16, n=16, kv_heads=8,
             heads=32, rot=128, style="half", fused_qkv=True, max_ctx=8192),
        # five sequences' prefill chunks together, three quarters of each head rotated
        dict(name="append_int2_chunks_4099", op="append", cache="int2", batch=5, n=4099,
             kv_heads=8, heads=32, rot=96, style="interleaved", fused_qkv=True, max_ctx=8192),
        # a large ragged batch's decode step into the BF16 cache
        dict(name="append_bf16_step_64", op="append", cache="bf16", batch=64, n=64, kv_heads=8,
             heads=32, rot=128, style="half", fused_qkv=True, max_ctx=8192),
        # a whole long prompt into the BF16 cache
        dict(name="append_bf16_prompt_32767", op="append", cache="bf16", batch=1, n=32767,
             kv_heads=8, heads=32, rot=128, style="half", fused_qkv=True, max_ctx=32768),
        # drafts of five tokens being verified, eight sequences
        dict(name="prefill_int2_verify_8x5", op="prefill", cache="int2", batch=8, n=40, heads=32,
             kv_heads=8, ctx=8192, mix="even"),
        # continuous batching: sixteen sequences decode one token each beside one prompt chunk
        dict(name="prefill_int2_mixed_17", op="prefill", cache="int2", batch=17, n=1037, heads=32,
             kv_heads=8, ctx=8192, mix="one_long"),
        # the last chunk of a 32K prompt
        dict(name="prefill_int2_4k_at_32k", op="prefill", cache="int2", batch=1, n=4096, heads=32,
             kv_heads=8, ctx=32768, mix="even"),
        # two whole prompts of odd length into empty BF16 caches
        dict(name="prefill_bf16_2x4093", op="prefill", cache="bf16", batch=2, n=8186, heads=32,
             kv_heads=8, ctx=4093, mix="even"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "table", "append", "append", "prefill", "prefill", "prefill"])
    if op == "rope":
        return dict(op=op, n=_log(rng, 1, 8191), heads=rng.choice([1, 4, 8, 16, 32]),
                    rot=rng.choice([128, 128, 96, 64, 32, 2 * rng.randint(1, 64)]),
                    style=rng.choice(["half", "interleaved"]), inverse=rng.random() < 0.5,
                    fused_qkv=rng.random() < 0.5, table_len=_log(rng, 8192, 65536))
    if op == "table":
        return dict(op=op, table_len=_log(rng, 100, 131072), rot=2 * rng.randint(2, 64),
                    kind=rng.choice(["none", "linear", "ntk", "yarn", "banded"]),
                    base=rng.choice([1e4, 5e5, 1e6]), factor=rng.choice([2.0, 4.0, 8.0]),
                    orig_len=rng.choice([4096, 8192, 32768]))
    g = rng.choice([1, 2, 4])
    hkv = rng.choice([1, 2, 3, 5, 8])
    cache = rng.choice(["int2", "bf16"])
    batch = _log(rng, 1, 32)
    if op == "append":
        n = max(batch, _log(rng, 1, 4099 if cache == "int2" else 16384))
        return dict(op=op, cache=cache, batch=batch, n=n, kv_heads=hkv, heads=hkv * g,
                    rot=rng.choice([128, 96, 64, 2 * rng.randint(1, 64)]),
                    style=rng.choice(["half", "interleaved"]), fused_qkv=rng.random() < 0.5,
                    max_ctx=max(n, _log(rng, 512, 8192)))
    ctx = _log(rng, 17, 16384)
    n = max(batch, min(batch * ctx, _log(rng, 1, 4096)))
    return dict(op=op, cache=cache, batch=batch, n=n, heads=hkv * g, kv_heads=hkv, ctx=ctx,
                mix=rng.choice(["even", "one_long", "ragged"]))


def _split(case):
    """New tokens of each sequence (they add up to n), and its context after them."""
    b, n = case["batch"], case["n"]
    top = case["ctx"] if case["op"] == "prefill" else case["max_ctx"]
    mix = case.get("mix", "even")
    if mix == "one_long" and b > 1 and n - (b - 1) <= top:
        new = [1] * (b - 1) + [n - (b - 1)]
    elif mix == "ragged" and b > 1:
        w = [1.0 + 3.0 * ((7 * i) % b) / b for i in range(b)]
        new = [min(top, max(1, int(n * x / sum(w)))) for x in w]
        for i in range(b):
            new[i] = min(top, new[i] + n - sum(new)) if sum(new) < n else new[i]
        i = 0
        while sum(new) > n:
            new[i % b] -= 1 if new[i % b] > 1 else 0
            i += 1
    else:
        new = [n // b + (1 if i < n % b else 0) for i in range(b)]
    # contexts between the new tokens alone and the whole length, the first one the longest
    lens = [max(new[i], top - (top - new[i]) * ((3 * i) % b) // (2 * b)) for i in range(b)]
    return new, lens


def work(case):
    op = case["op"]
    if op == "table":
        return {"bytes": 4 * case["table_len"] * case["rot"],
                "flops": 20 * case["table_len"] * case["rot"]}
    if op == "rope":
        n, hd = case["n"], case["heads"] * D
        return {"bytes": n * (2 * hd * 2 + 4 * case["rot"] + 4),
                "flops": n * case["heads"] * case["rot"] * 3}
    if op == "append":
        n, hkv = case["n"], case["kv_heads"]
        read = n * (2 * hkv * D * 2 + 4 * case["rot"] + 8)
        if case["cache"] == "bf16":
            return {"bytes": read + n * hkv * 2 * D * 2, "flops": n * hkv * case["rot"] * 3}
        return {"bytes": read + n * hkv * 72 + 2 * hkv * D * D * 4,
                "flops": n * hkv * (2 * 2 * D * D + case["rot"] * 3)}
    new, lens = _split(case)
    h, hkv = case["heads"], case["kv_heads"]
    per = 72 if case["cache"] == "int2" else 512
    seen = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(new, lens))
    turn = case["n"] * h * D * D * 4 if case["cache"] == "int2" else 0
    return {"bytes": 2 * case["n"] * h * D * 2 + sum(lens) * hkv * per
            + (2 * hkv * D * D * 4 if case["cache"] == "int2" else 0),
            "flops": 4 * D * h * seen + turn}


# ---- inputs -------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _frequencies(rot, kind="none", base=1e4, factor=1.0, orig_len=8192):
    """Radians per position of each pair, in 64 bits, and the factor on cos and sin."""
    i = np.arange(rot // 2, dtype=np.float64)
    if kind == "ntk":
        base = base * factor ** (rot / (rot - 2))
    inv = base ** (-2.0 * i / rot)
    amp = 1.0
    if kind == "linear":
        inv = inv / factor
    elif kind == "yarn":      # beta_fast 32, beta_slow 1
        def pair(turns):
            return rot * math.log(orig_len / (turns * 2 * math.pi)) / (2 * math.log(base))
        low = max(math.floor(pair(32.0)), 0)
        high = min(math.ceil(pair(1.0)), rot - 1)
        ramp = np.clip((i - low) / max(high - low, 1e-3), 0.0, 1.0)
        inv = inv / factor * ramp + inv * (1.0 - ramp)
        amp = 0.1 * math.log(factor) + 1.0
    elif kind == "banded":    # low factor 1, high factor 4
        turns = orig_len * inv / (2 * math.pi)
        smooth = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        inv = (1.0 - smooth) * inv / factor + smooth * inv
    return inv, amp


def _table(table_len, rot, **kw):
    inv, amp = _frequencies(rot, **kw)
    a = (torch.arange(table_len, device="cuda", dtype=torch.float64)[:, None]
         * torch.from_numpy(inv).cuda()[None])
    return (torch.cat([a.cos(), a.sin()], 1) * amp).float()


def _pages(g, lens, extra=7):
    """Shuffled page table [batch, max_pages] (-1 where a sequence has no page), pool pages."""
    need = [(c + PAGE - 1) // PAGE for c in lens]
    total = sum(need) + extra
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    pt = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        pt[b, :m] = order[at:at + m]
        at += m
    return pt, total


def _rotation(g, hkv):
    """[2, hkv, 128, 128] orthogonal: four reflections of each head."""
    r = torch.eye(D, device="cuda", dtype=torch.float64).repeat(2, hkv, 1, 1)
    for _ in range(4):
        v = _randn(g, 2, hkv, D, 1).double()
        v = v / v.square().sum(2, keepdim=True).sqrt()
        r = r - 2.0 * (r * v.transpose(2, 3)).sum(3, keepdim=True) * v.transpose(2, 3)
    return r.float().contiguous()


def _int2_pool(g, pages, hkv):
    """Records whose codes and scales are those of normal keys and values."""
    n = pages * hkv
    pool = torch.empty(n, INT2_REC, dtype=torch.uint8, device="cuda")
    u = torch.randint(0, 20, (n, 1024, 4), generator=g, device="cuda", dtype=torch.uint8)
    c = (u > 0).to(torch.uint8) + (u > 9).to(torch.uint8) + (u > 18).to(torch.uint8)
    pool[:, :1024] = c[..., 0] | (c[..., 1] << 2) | (c[..., 2] << 4) | (c[..., 3] << 6)
    s = (torch.rand(n, 8, 2, 2, 1, generator=g, device="cuda") * 0.4 + 0.8) * torch.tensor(
        [3.2, 1.6], device="cuda").view(1, 1, 2, 1, 1)
    z = -1.5 * s + 0.1 * s * _randn(g, n, 8, 2, 2, 1)
    pool[:, 1024:] = torch.cat([s, z], 4).half().view(torch.uint8).reshape(n, 128)
    return pool.reshape(-1)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = dict(case=case)
    if op == "table":
        # the frequencies' base is a weight of the model: another seed, another model
        st["spec"] = dict(kind=case["kind"], base=case["base"] * (1.0 + (seed % 97) / 97.0),
                          factor=case["factor"], orig_len=case["orig_len"])
        if own:
            from rotated_int2_kv_kvq_gb300 import kvq as K
            st["table"] = torch.empty(case["table_len"], case["rot"], device="cuda")
            st["scaling"] = K.make_rope_scaling(**st["spec"])
        return st
    hkv = case.get("kv_heads", 1)
    heads = case["heads"]
    if op == "rope":
        n = case["n"]
        total = heads + 2 if case["fused_qkv"] else heads
        st["table"] = _table(case["table_len"], case["rot"])
        st["positions"] = torch.randint(0, case["table_len"], (n,), generator=g, device="cuda",
                                        dtype=torch.int32)
        st["x"] = _randn(g, n, total, D).to(torch.bfloat16)[:, :heads]
        st["y"] = torch.empty(n, heads, D, dtype=torch.bfloat16, device="cuda")
    elif op == "append":
        n = case["n"]
        new, lens = _split(case)
        st["pt"], st["pages"] = _pages(g, lens)
        st["seq_idx"] = torch.cat([torch.full((m,), b, dtype=torch.int32) for b, m in
                                   enumerate(new)]).cuda()
        st["positions"] = torch.cat([torch.arange(c - m, c, dtype=torch.int32) for m, c in
                                     zip(new, lens)]).cuda()
        st["table"] = _table(max(lens), case["rot"])
        if case["fused_qkv"]:
            qkv = _randn(g, n, heads + 2 * hkv, D).to(torch.bfloat16)
            st["k"], st["v"] = qkv[:, heads:heads + hkv], qkv[:, heads + hkv:]
        else:
            st["k"] = _randn(g, n, hkv, D).to(torch.bfloat16)
            st["v"] = _randn(g, n, hkv, D).to(torch.bfloat16)
        st["R"], st["mu"] = _rotation(g, hkv), 2.0 * _randn(g, hkv, D)
        if case["cache"] == "int2":
            st["pool"] = _int2_pool(g, st["pages"], hkv)
        else:
            st["pool"] = _randn(g, st["pages"] * hkv * BF16_REC // 2).to(torch.bfloat16).view(
                torch.uint8)
    else:
        new, lens = _split(case)
        st["new"], st["lens"] = new, lens
        st["pt"], st["pages"] = _pages(g, lens)
        st["cu_q"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
        st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["q"] = _randn(g, case["n"], heads, D).to(torch.bfloat16)
        st["R"], st["mu"] = _rotation(g, hkv), torch.zeros(hkv, D, device="cuda")
        if case["cache"] == "int2":
            st["pool"] = _int2_pool(g, st["pages"], hkv)
        else:
            st["pool"] = (1.5 * _randn(g, st["pages"] * hkv * BF16_REC // 2)).to(
                torch.bfloat16).view(torch.uint8)
    if op != "rope":
        st["places"] = _cuda(*(_int2_places() if case["cache"] == "int2" else _bf16_places()))
    if own:
        from rotated_int2_kv_kvq_gb300 import kvq as K
        st["h"] = K.kvq_create(K.make_layout(heads if op != "rope" else 1, hkv, CLIP_K, CLIP_V))
        if op != "rope":
            K.kvq_set_rotation(st["h"], st["R"], st["mu"])
        if op == "prefill":
            size = (K.kvq_prefill_workspace_bytes if case["cache"] == "int2"
                    else K.kvq_bf16_prefill_workspace_bytes)
            st["ws"] = torch.empty(size(st["h"], case["batch"], case["n"]), dtype=torch.uint8,
                                   device="cuda")
            st["out"] = torch.empty(case["n"], heads, D, dtype=torch.bfloat16, device="cuda")
        else:
            st["rope"] = K.make_rope(st["table"], case["style"])
    return st


# ---- the page records' layouts --------------------------------------------------------------------

def _int2_places():
    """For slot tau and element d: 16-bit word and bit of the key's and of the value's code, and
    the 16-bit words of their scale and zero."""
    tau, d = np.meshgrid(np.arange(PAGE), np.arange(D), indexing="ij")
    w, r = d >> 4, d & 15
    kw = 8 * (4 * (tau & 7) + ((r >> 1) & 3)) + 2 * (2 * (tau >> 3) + (r >> 3)) + (r & 1)
    vw = (256 + 8 * (4 * (r & 7) + ((tau & 7) >> 1)) + 2 * (2 * (tau >> 3) + (r >> 3))
          + (tau & 1))
    t = np.arange(PAGE)
    sc = 512 + 8 * (t & 7) + 2 * (t >> 3)
    return kw, vw, 2 * w, np.stack([sc, sc + 1, sc + 4, sc + 5], 1)


def _bf16_places():
    """For slot tau and element d: the element's place in a BF16 record, keys and values."""
    tau, d = np.meshgrid(np.arange(PAGE), np.arange(D), indexing="ij")
    w, r = d >> 4, d & 15
    k = (256 * w + 8 * (4 * (tau & 7) + ((r >> 1) & 3)) + 2 * ((tau >> 3) + 2 * (r >> 3))
         + (r & 1))
    v = (2048 + 256 * w + 8 * (4 * (r & 7) + ((tau & 7) >> 1))
         + 2 * (2 * (tau >> 3) + (r >> 3)) + (tau & 1))
    return k, v


def _cuda(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).long().cuda() for a in arrays]


def _read_cache(st, b, dtype):
    """Keys and values [kv_heads, length, 128] of sequence b as the cache holds them."""
    hkv, n = st["case"]["kv_heads"], st["lens"][b]
    ids = st["pt"][b, :(n + PAGE - 1) // PAGE].long()
    if st["case"]["cache"] == "bf16":
        rec = st["pool"].view(torch.bfloat16).view(st["pages"], hkv, BF16_REC // 2)[ids]
        kp, vp = st["places"]
        k, v = rec[..., kp].to(dtype), rec[..., vp].to(dtype)
    else:
        rec = st["pool"].view(torch.int16).view(st["pages"], hkv, INT2_REC // 2)[ids]
        kw, vw, bit, sc = st["places"]
        m = rec[..., sc].view(torch.float16).to(dtype)
        k = ((rec[..., kw].int() >> bit) & 3).to(dtype) * m[..., 0:1] + m[..., 1:2]
        v = ((rec[..., vw].int() >> bit) & 3).to(dtype) * m[..., 2:3] + m[..., 3:4]
    flat = [x.permute(1, 0, 2, 3).reshape(hkv, -1, D)[:, :n] for x in (k, v)]
    return flat


# ---- plain forms ----------------------------------------------------------------------------------

def _plain_rope(x, positions, table, rot, style, inverse=False):
    """Each product rounded to 32 bits, then their difference or sum, then bf16: the library's
    definition of the rotation."""
    cs = table[positions.long()][:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    s = -s if inverse else s
    f = x.float()
    lead, rest = f[..., :rot], f[..., rot:]
    if style == "half":
        a, b = lead[..., :rot // 2], lead[..., rot // 2:]
    else:
        a, b = lead[..., 0::2], lead[..., 1::2]
    p, q = a * c - b * s, b * c + a * s
    turned = torch.cat([p, q], -1) if style == "half" else torch.stack([p, q], -1).flatten(-2)
    return torch.cat([turned, rest], -1).to(torch.bfloat16)


def _plain_codes(x, r, clip):
    """INT2 codes, scale and zero of rows [n, kv_heads, 128].  The cache's format fixes the order
    of the rotation's sum and one rounding to 32 bits a step, because the stored bytes have to be
    the same whoever writes them: a product of two 32-bit numbers is exact in 64."""
    a, xd, rd = torch.zeros_like(x), x.double(), r.double()
    for j in range(D):
        a = torch.addcmul(a.double(), xd[..., j:j + 1], rd[:, j]).float()
    hi = clip * a.amax(-1, keepdim=True)
    lo = clip * a.amin(-1, keepdim=True)
    three = torch.full_like(hi, 3.0)       # a tensor: an IEEE division, not a product
    s, z = ((hi - lo) / three).half(), lo.half()
    sf, zf = s.float(), z.float()
    code = torch.round((a - zf) / torch.where(sf == 0, torch.ones_like(sf), sf)).clamp(0, 3)
    return torch.where(sf == 0, torch.zeros_like(code), code).int(), s, z


def _plain_append(st):
    c, hkv = st["case"], st["case"]["kv_heads"]
    k = _plain_rope(st["k"], st["positions"], st["table"], c["rot"], c["style"])
    pos, n = st["positions"].long(), c["n"]
    page = st["pt"][st["seq_idx"].long(), pos // PAGE].long()
    rec = page[:, None] * hkv + torch.arange(hkv, device="cuda")
    slot = pos % PAGE
    if c["cache"] == "bf16":
        pool = st["pool"].view(torch.bfloat16)
        kp, vp = st["places"]
        base = rec[..., None] * (BF16_REC // 2)
        pool[base + kp[slot][:, None]] = k
        pool[base + vp[slot][:, None]] = st["v"]
        return {"pool": pool}
    pool = st["pool"].view(torch.int16)
    kw, vw, bit, sc = st["places"]
    base = rec[..., None] * (INT2_REC // 2)
    for x, place, which, clip in ((k.float() - st["mu"], kw, 0, CLIP_K),
                                  (st["v"].float(), vw, 1, CLIP_V)):
        codes, s, z = _plain_codes(x, st["R"][which], clip)
        # eight codes make a 16-bit word: elements 16 apart share one
        words = (codes << bit[0]).view(n, hkv, 8, 16).sum(2)
        words = torch.where(words > 32767, words - 65536, words).short()
        pool[base + place[slot][:, None, :16]] = words
        meta = torch.cat([s, z], -1).view(torch.int16)
        pool[base + sc[slot][:, None, 2 * which:2 * which + 2]] = meta
    return {"pool": st["pool"]}


def _plain_prefill(st):
    c = st["case"]
    hkv, g = c["kv_heads"], c["heads"] // c["kv_heads"]
    out = torch.empty(c["n"], c["heads"], D, dtype=torch.bfloat16, device="cuda")
    at = 0
    for b, (n, length) in enumerate(zip(st["new"], st["lens"])):
        k, v = _read_cache(st, b, torch.float32)
        q = st["q"][at:at + n].float().view(n, hkv, g, D).permute(1, 2, 0, 3).reshape(hkv, g * n, D)
        if c["cache"] == "int2":
            q = torch.matmul(q, st["R"][0])
        s = torch.matmul(q, k.transpose(1, 2)).view(hkv, g, n, length)
        s *= 1.0 / math.sqrt(D)
        row = torch.arange(length - n, length, device="cuda")[:, None]
        s.masked_fill_(torch.arange(length, device="cuda") > row, -math.inf)
        s = s.sub_(s.amax(-1, keepdim=True)).exp_()
        total = s.sum(-1, keepdim=True)
        o = torch.matmul(s.view(hkv, g * n, length), v).view(hkv, g, n, D) / total
        if c["cache"] == "int2":
            o = torch.matmul(o.view(hkv, g * n, D), st["R"][1].transpose(1, 2)).view(hkv, g, n, D)
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, c["heads"], D).to(torch.bfloat16)
        at += n
    return out


def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        if op == "table":
            return _table(c["table_len"], c["rot"], **st["spec"])
        if op == "rope":
            return _plain_rope(st["x"], st["positions"], st["table"], c["rot"], c["style"],
                               c["inverse"])
        return _plain_append(st) if op == "append" else _plain_prefill(st)
    from rotated_int2_kv_kvq_gb300 import kvq as K
    if op == "table":
        K.kvq_rope_table(st["table"], st["scaling"])
        return st["table"]
    if op == "rope":
        K.kvq_rope(st["h"], st["x"], st["y"], st["positions"], st["rope"], inverse=c["inverse"])
        return st["y"]
    int2 = c["cache"] == "int2"
    if op == "append":
        fn = K.kvq_append_rope if int2 else K.kvq_bf16_append_rope
        fn(st["h"], st["pool"], st["pages"], st["k"], st["v"], st["seq_idx"], st["positions"],
           st["pt"], st["rope"])
        return {"pool": st["pool"] if int2 else st["pool"].view(torch.bfloat16)}
    fn = K.kvq_prefill if int2 else K.kvq_bf16_prefill
    fn(st["h"], st["pool"], st["pages"], st["q"], st["cu_q"], st["pt"], st["seq_lens"], st["out"],
       st["ws"])
    return st["out"]


# ---- in 64 bits -----------------------------------------------------------------------------------

def exact(case, seed):
    """From the definitions, in 64 bits: rotations as complex products, attention over the cache's
    entries turned back to the plain basis, one KV head at a time."""
    if case["op"] == "append" and case["cache"] == "int2":
        return None       # bytes: codes are whole numbers, and compared as such
    st = prepare(case, seed)
    if case["op"] == "table":
        inv, amp = _frequencies(case["rot"], **st["spec"])
        out = np.empty((case["table_len"], case["rot"]))
        turn = np.exp(1j * np.outer(np.arange(case["table_len"]), inv))
        out[:, :case["rot"] // 2], out[:, case["rot"] // 2:] = amp * turn.real, amp * turn.imag
        return torch.from_numpy(out)
    if case["op"] in ("rope", "append"):
        rot, half = case["rot"], case["rot"] // 2
        x = (st["x"] if case["op"] == "rope" else st["k"]).double()
        t = st["table"].double()[st["positions"].long()]
        turn = torch.complex(t[:, :half], t[:, half:])[:, None]
        if case.get("inverse"):
            turn = turn.conj()
        first = slice(0, half) if case["style"] == "half" else slice(0, rot, 2)
        second = slice(half, rot) if case["style"] == "half" else slice(1, rot, 2)
        w = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = w.real, w.imag
        if case["op"] == "rope":
            return x
        hkv, pos = case["kv_heads"], st["positions"].long()
        pool = st["pool"].view(torch.bfloat16).double().view(st["pages"], hkv, BF16_REC // 2)
        page, slot = st["pt"][st["seq_idx"].long(), pos // PAGE].long(), pos % PAGE
        for values, place in zip((x, st["v"].double()), st["places"]):
            for kv in range(hkv):
                pool[page[:, None], kv, place[slot]] = values[:, kv]
        return {"pool": pool.view(-1)}
    hkv, g = case["kv_heads"], case["heads"] // case["kv_heads"]
    out = torch.empty(case["n"], case["heads"], D, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, length) in enumerate(zip(st["new"], st["lens"])):
        keys, values = _read_cache(st, b, torch.float64)
        hidden = torch.ones(n, length, device="cuda", dtype=torch.bool).triu(length - n + 1)
        for kv in range(hkv):
            k, v = keys[kv], values[kv]
            if case["cache"] == "int2":
                k = k @ st["R"][0, kv].double().T
                v = v @ st["R"][1, kv].double().T
            for h in range(kv * g, kv * g + g):
                s = st["q"][at:at + n, h].double() @ k.T / math.sqrt(D)
                out[at:at + n, h] = torch.softmax(s.masked_fill(hidden, -math.inf), 1) @ v
        at += n
    return out
