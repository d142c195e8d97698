"""The 8-bit paged cache, its attention, and the norms of queries and keys, as cases that can be
timed.

Four operators that carry tokens from the fused projection into a cache held in 8 bits and back
out through attention, each in its plain form (elementary torch operations) and, with ``own``
true, through the library's entry points:

- ``norm``    : root-mean-square norm of each query and key head and the rotation by the token's
  position in one pass, and its backward pass (``kvq_norm_rope``, ``kvq_norm_rope_backward``);
- ``store``   : keys and values into the 8-bit cache, one scale for each page and KV head, and
  positions of it read back (``kvq_fp8_append``, ``kvq_fp8_read``);
- ``decode``  : attention of one token a sequence over that cache, all of it or a sliding window
  and a few first tokens (``kvq_fp8_decode``);
- ``prefill`` : the same of many new tokens a sequence (``kvq_fp8_prefill``).

The cache's definition.  A record holds 16 tokens of one KV head: 8-bit floating-point codes
(four exponent bits, three of mantissa, largest 448) of K and of V, and a power of two for each,
s = 2^e; an entry is code * s.  A call that appends to a page gives K and V of each head the e of
    max(e of the page, e of the new tokens),  e of the new tokens = the least e >= -100 with
    max |x| <= 448 * 2^e,
rounds the new tokens to the nearest code (ties to even) and, where e grew, the older ones again
from what they stood for.  A call that writes a page's first slot begins the page: what it held
counts no more.  Everything is made from the seed alone.
"""
import math

import numpy as np
import torch

own = False

D, PAGE = 128, 16
REC = 4112                     # bytes of a record: 2048 K codes, 2048 V codes, two scales, flags
EPS = 1e-6


# ---- cases --------------------------------------------------------------------------------------

def listed():
    """Twelve cases.  32 query heads over 8 KV heads, batch 16, 32K contexts, the 64-sequence
    ragged batch and the 1K context of one KV head are this library's benchmark shapes; the
    others are generic."""
    return [
        # one decode step of 16 sequences, queries and keys inside the fused projection's output
        dict(name="norm_step_16", op="norm", back=False, n=16, heads=32, kv_heads=8, rot=128,
             style="half", table_len=32768, fused_qkv=True),
        # a long prompt's
        dict(name="norm_chunk_8191", op="norm", back=False, n=8191, heads=32, kv_heads=8, rot=128,
             style="half", table_len=32768, fused_qkv=True),
        # training on a short sample, half of each head rotated, pairs side by side
        dict(name="norm_back_257", op="norm", back=True, n=257, heads=8, kv_heads=2, rot=64,
             style="interleaved", table_len=8192, fused_qkv=False),
        # training on a packed batch
        dict(name="norm_back_4099", op="norm", back=True, n=4099, heads=32, kv_heads=8, rot=128,
             style="half", table_len=8192, fused_qkv=False),
        # one token of each of 64 sequences, and the last block of each read back
        dict(name="store_step_64", op="store", batch=64, n=64, heads=32, kv_heads=8, ctx=8192,
             mix="even", read="tail", fused_qkv=False),
        # three prompts of 32767 tokens together, behind older tokens; all of it handed on
        dict(name="store_prompts_32767", op="store", batch=3, n=32767, heads=32, kv_heads=8,
             ctx=16384, mix="ragged", read="all", fused_qkv=True),
        # one short context of one KV head: latency
        dict(name="decode_1x1k", op="decode", batch=1, heads=4, kv_heads=1, ctx=1024, ragged=False,
             window=0, sinks=0),
        # a decode step of 16 sequences at 32K
        dict(name="decode_16x32k", op="decode", batch=16, heads=32, kv_heads=8, ctx=32768,
             ragged=False, window=0, sinks=0),
        # a step of 64 ragged sequences up to 64K, of which a layer sees 4096 tokens and four first
        dict(name="decode_window_64", op="decode", batch=64, heads=32, kv_heads=8, ctx=65536,
             ragged=True, window=4096, sinks=4),
        # eight sequences verify five drafted tokens each
        dict(name="prefill_verify_8x5", op="prefill", batch=8, n=40, heads=32, kv_heads=8,
             ctx=8192, mix="even", window=0, sinks=0),
        # a prompt of odd length through a layer that sees 1024 tokens and four first
        dict(name="prefill_window_8191", op="prefill", batch=1, n=8191, heads=32, kv_heads=8,
             ctx=8191, mix="even", window=1024, sinks=4),
        # the last chunk of a 32K prompt
        dict(name="prefill_4k_at_32k", op="prefill", batch=1, n=4096, heads=32, kv_heads=8,
             ctx=32768, mix="even", window=0, sinks=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "store", "store", "decode", "decode", "decode", "prefill",
                     "prefill", "prefill"])
    g = rng.choice([1, 2, 4])
    hkv = rng.choice([1, 2, 3, 5, 8])
    if op == "norm":
        return dict(op=op, back=rng.random() < 0.5, n=_log(rng, 1, 8191), heads=hkv * g,
                    kv_heads=hkv, rot=rng.choice([128, 128, 64, 2 * rng.randint(1, 64)]),
                    style=rng.choice(["half", "interleaved"]), table_len=_log(rng, 8192, 65536),
                    fused_qkv=rng.random() < 0.5)
    window, sinks = rng.choice([(0, 0), (_log(rng, 1, 8192), rng.choice([0, 1, 4, 64]))])
    batch = _log(rng, 1, 64)
    if op == "decode":
        ctx = min(_log(rng, 1, 65536), 16 * 32768 // batch)
        return dict(op=op, batch=batch, heads=hkv * g, kv_heads=hkv, ctx=ctx,
                    ragged=rng.random() < 0.5, window=window, sinks=sinks)
    if op == "store":
        n = max(batch, _log(rng, 1, 16384))
        ctx = min(max(n, _log(rng, 17, 8192)), 3 * 16384 // batch)
        return dict(op=op, batch=batch, n=n, heads=hkv * g, kv_heads=hkv, ctx=ctx,
                    mix=rng.choice(["even", "one_long", "ragged"]),
                    read=rng.choice(["tail", "all"]), fused_qkv=rng.random() < 0.5)
    batch = _log(rng, 1, 32)
    ctx = _log(rng, 17, 16384)
    n = max(batch, min(batch * ctx, _log(rng, 1, 4096)))
    return dict(op=op, batch=batch, n=n, heads=hkv * g, kv_heads=hkv, ctx=ctx,
                mix=rng.choice(["even", "one_long", "ragged"]), window=window, sinks=sinks)


def _split(case):
    """New tokens of each sequence (they add up to n), and its context after them."""
    b, n, top, mix = case["batch"], case["n"], case["ctx"], case["mix"]
    if mix == "one_long" and b > 1 and n - (b - 1) <= top:
        new = [1] * (b - 1) + [n - (b - 1)]
    else:
        w = [1.0 + (3.0 * ((7 * i) % b) / b if mix == "ragged" else 0.0) for i in range(b)]
        new = [min(top, max(1, int(n * x / sum(w)))) for x in w]
        i = 0
        while sum(new) != n:            # what rounding left over, or took too much
            d = max(-1, min(1, n - sum(new)))
            if 1 <= new[i % b] + d <= top:
                new[i % b] += d
            i += 1
    # contexts between the new tokens alone and the whole length, the first one the longest
    lens = [max(new[i], top - (top - new[i]) * ((3 * i) % b) // (2 * b)) for i in range(b)]
    return new, lens


def _lens(case):
    """Contexts of a decode step: all alike, or between a sixty-fourth of the longest and it."""
    b, top = case["batch"], case["ctx"]
    if not case["ragged"]:
        return [top] * b
    return [max(1, int(round(top * 64.0 ** (-((5 * i) % b) / b)))) for i in range(b)]


def _sees(case, p):
    """How many positions the token at position p attends to."""
    w, s = case["window"], case["sinks"]
    return p + 1 if w == 0 else min(p + 1, w) + max(0, min(s, p + 1 - w))


def work(case):
    op, h, hkv = case["op"], case["heads"], case["kv_heads"]
    if op == "norm":
        rows = case["n"] * (h + hkv)
        small = case["n"] * (4 * case["rot"] + 4) + 2 * D * 4 * (2 if case["back"] else 1)
        return {"bytes": rows * D * 2 * (3 if case["back"] else 2) + small,
                "flops": rows * D * (20 if case["back"] else 8)}
    per = REC / PAGE                              # bytes a token and KV head
    if op == "store":
        new, lens = _split(case)
        back = _read_counts(case, new, lens)
        # the new tokens read and written once (a page that goes on also has its scales read),
        # the read positions' codes read and their 16-bit values written
        return {"bytes": case["n"] * hkv * (2 * D * 2 + per) + sum(back) * hkv * (per + 2 * D * 2),
                "flops": (case["n"] + sum(back)) * hkv * 2 * D * 2}
    if op == "decode":
        seen = sum(_sees(case, c - 1) for c in _lens(case))
        return {"bytes": seen * hkv * per + case["batch"] * h * D * 6, "flops": 4 * D * h * seen}
    new, lens = _split(case)
    pairs = held = 0
    for n, c in zip(new, lens):
        pairs += sum(_sees(case, p) for p in range(c - n, c))
        first = 0 if case["window"] == 0 else max(0, c - n + 1 - case["window"])
        held += c - first + min(case["sinks"], first)
    return {"bytes": 2 * case["n"] * h * D * 2 + held * hkv * per, "flops": 4 * D * h * pairs}


def _read_counts(case, new, lens):
    return list(lens) if case["read"] == "all" else [min(c, PAGE) for c in lens]


# ---- inputs -------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _i32(values):
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


def _cu(counts):
    return _i32([0] + [int(x) for x in np.cumsum(counts)])


def _table(table_len, rot):
    """cos and sin of every position, frequencies 10000^(-2i / rot)."""
    inv = 1e4 ** (-2.0 * np.arange(rot // 2, dtype=np.float64) / rot)
    a = (torch.arange(table_len, device="cuda", dtype=torch.float64)[:, None]
         * torch.from_numpy(inv).cuda()[None])
    return torch.cat([a.cos(), a.sin()], 1).float()


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


def _pool(g, pages, hkv):
    """Records of normal keys (of two sizes) and values, each on one of three scales."""
    n = pages * hkv
    pool = torch.zeros(n, REC, dtype=torch.uint8, device="cuda")
    e = torch.randint(-7, -4, (n, 2), generator=g, device="cuda")
    for which in range(2):
        x = _randn(g, n, 2048) * (1.5 if which == 0 else 1.0)
        code = (x * torch.exp2(-e[:, which:which + 1].float())).clamp_(-448, 448)
        pool[:, 2048 * which:2048 * which + 2048] = code.to(torch.float8_e4m3fn).view(torch.uint8)
    pool[:, 4096:4104] = torch.exp2(e.float()).contiguous().view(torch.uint8)
    return pool.view(-1)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = dict(case=case)
    h, hkv = case["heads"], case["kv_heads"]
    if op == "norm":
        n = case["n"]
        st["table"] = _table(case["table_len"], case["rot"])
        st["positions"] = torch.randint(0, case["table_len"], (n,), generator=g, device="cuda",
                                        dtype=torch.int32)
        x = (2.0 * _randn(g, n, h + 2 * hkv, D)).to(torch.bfloat16)
        st["q"], st["k"] = x[:, :h], x[:, h:h + hkv]
        if not case["fused_qkv"]:
            st["q"], st["k"] = st["q"].contiguous(), st["k"].contiguous()
        st["wq"], st["wk"] = (1.0 + 0.3 * _randn(g, D) for _ in range(2))
        if case["back"]:
            st["dq"] = _randn(g, n, h, D).to(torch.bfloat16)
            st["dk"] = _randn(g, n, hkv, D).to(torch.bfloat16)
    else:
        if op == "decode":
            lens = _lens(case)
            st["q"] = _randn(g, case["batch"], h, D).to(torch.bfloat16)
        else:
            st["new"], lens = _split(case)
            st["cu"] = _cu(st["new"])
        st["lens"] = lens
        st["pt"], st["pages"] = _pages(g, lens)
        st["pool"] = _pool(g, st["pages"], hkv)
        st["seq_lens"] = _i32(lens)
        st["places"] = _places()
        if op == "prefill":
            st["q"] = _randn(g, case["n"], h, D).to(torch.bfloat16)
        if op == "store":
            x = _randn(g, case["n"], h + 2 * hkv, D).to(torch.bfloat16)
            st["k"], st["v"] = x[:, h:h + hkv], x[:, h + hkv:]
            if not case["fused_qkv"]:
                st["k"], st["v"] = st["k"].contiguous(), st["v"].contiguous()
            st["back"] = _read_counts(case, st["new"], lens)
            st["cu_back"] = _cu(st["back"])
    if own:
        from rotated_int2_kv_kvq_gb300 import kvq as K
        st["h"] = K.kvq_create(K.make_layout(h, hkv))

        def buffer(size):
            return torch.empty(size, dtype=torch.uint8, device="cuda")

        if op == "norm":
            n = case["n"]
            st["rope"] = K.make_rope(st["table"], case["style"])
            st["yq"] = torch.empty(n, h, D, dtype=torch.bfloat16, device="cuda")
            st["yk"] = torch.empty(n, hkv, D, dtype=torch.bfloat16, device="cuda")
            if case["back"]:
                st["dwq"], st["dwk"] = (torch.empty(D, device="cuda") for _ in range(2))
                st["ws"] = buffer(K.kvq_norm_rope_backward_workspace_bytes(st["h"], n))
        elif op == "store":
            st["ko"], st["vo"] = (torch.empty(sum(st["back"]), hkv, D, dtype=torch.bfloat16,
                                              device="cuda") for _ in range(2))
        elif op == "decode":
            st["ws"] = buffer(K.kvq_fp8_workspace_bytes(st["h"], case["batch"]))
            st["out"] = torch.empty(case["batch"], h, D, device="cuda")
        else:
            st["ws"] = buffer(K.kvq_fp8_prefill_workspace_bytes(st["h"], case["batch"], case["n"]))
            st["out"] = torch.empty(case["n"], h, D, dtype=torch.bfloat16, device="cuda")
    return st


# ---- the page record's layout --------------------------------------------------------------------

def _places():
    """For slot tau and element d: the code's byte in a record, keys and values [16, 128]."""
    tau, d = np.meshgrid(np.arange(PAGE), np.arange(D), indexing="ij")
    w, r = d >> 4, d & 15
    k = (512 * (w >> 1) + 16 * (4 * (tau & 7) + ((r >> 1) & 3)) + 4 * ((tau >> 3) + 2 * (r >> 3))
         + 2 * (w & 1) + (r & 1))
    v = (2048 + 512 * (w >> 1) + 16 * (4 * (r & 7) + ((tau & 7) >> 1))
         + 4 * (2 * (w & 1) + (r >> 3)) + 2 * (tau >> 3) + (tau & 1))
    return [torch.from_numpy(np.ascontiguousarray(x)).long().cuda() for x in (k, v)]


def _entries(st, at, dtype=torch.float32):
    """Keys and values [..., kv_heads, 16, 128] of the pages `at` (ids)."""
    rec = st["pool"].view(st["pages"], st["case"]["kv_heads"], REC)[at]
    scale = rec[..., 4096:4104].contiguous().view(torch.float32)
    got = []
    for which, place in enumerate(st["places"]):
        code = rec[..., place].view(torch.float8_e4m3fn).to(dtype)
        got.append(code * scale[..., which, None, None].to(dtype))
    return got


# ---- plain forms ----------------------------------------------------------------------------------

def _turn(x, positions, table, rot, style, back=False):
    """Pairs of the first `rot` elements turned by the angles of the positions (back: the
    transposed map)."""
    cs = table[positions.long()][:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    s = -s if back else s
    lead, rest = x[..., :rot], x[..., rot:]
    if style == "half":
        a, b = lead[..., :rot // 2], lead[..., rot // 2:]
    else:
        a, b = lead[..., 0::2], lead[..., 1::2]
    p, q = a * c - b * s, b * c + a * s
    turned = torch.cat([p, q], -1) if style == "half" else torch.stack([p, q], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _plain_norm(st):
    """y = turn(x w / sqrt(mean(x^2) + eps)), or the gradients of x and of w."""
    c, out = st["case"], {}
    how = (st["positions"], st["table"], c["rot"], c["style"])
    for name, w in (("q", st["wq"]), ("k", st["wk"])):
        x = st[name].float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        if not c["back"]:
            out[name] = _turn(x * r * w, *how).to(torch.bfloat16)
            continue
        dn = _turn(st["d" + name].float(), *how, back=True)
        xh, g = x * r, dn * w
        out["d" + name] = (r * (g - xh * (g * xh).mean(-1, keepdim=True))).to(torch.bfloat16)
        out["dw" + name] = (dn * xh).double().sum((0, 1)).float()
    return out


def _plain_store(st):
    """Appends the tokens, then reads positions back."""
    c, hkv = st["case"], st["case"]["kv_heads"]
    pool = st["pool"].view(st["pages"], hkv, REC)
    new = st["cu"].diff().long()
    seq = torch.repeat_interleave(new)
    pos = torch.arange(c["n"], device="cuda") + (st["seq_lens"].long() - st["cu"][1:].long())[seq]
    page, slot = st["pt"][seq, pos // PAGE].long(), pos % PAGE
    pages, mine = torch.unique(page, return_inverse=True)      # the pages that get a token
    m = pages.numel()
    begun = torch.zeros(m, dtype=torch.bool, device="cuda").index_fill_(0, mine[slot == 0], True)
    rec = pool[pages]
    old = rec[..., 4096:4104].contiguous().view(torch.float32)
    old = torch.where(begun[:, None, None], torch.full_like(old, 2.0 ** -100), old)
    scales = []
    for which, (x, place) in enumerate(zip((st["k"].float(), st["v"].float()), st["places"])):
        top = torch.zeros(m, hkv, device="cuda").scatter_reduce_(
            0, mine[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
        mant, ex = torch.frexp(top)                       # top = mant * 2^ex; 448 = 0.875 * 2^9
        e = torch.where(top > 0, ex - 8 - (mant <= 0.875).int(), -100).clamp_(min=-100)
        s = torch.maximum(torch.exp2(e.float()), old[..., which])
        held = rec[..., place].view(torch.float8_e4m3fn).float() * (old[..., which] / s)[..., None, None]
        held = torch.where(begun[:, None, None, None], torch.zeros_like(held), held)
        held[mine, :, slot] = x / s[mine][..., None]
        rec[..., place] = held.to(torch.float8_e4m3fn).view(torch.uint8)
        scales.append(s)
    rec[..., 4096:4104] = torch.stack(scales, -1).contiguous().view(torch.uint8)
    pool[pages] = rec
    back = st["cu_back"].diff().long()
    total = sum(st["back"])
    seq = torch.repeat_interleave(back, output_size=total)
    pos = torch.arange(total, device="cuda") + (st["seq_lens"].long()
                                                - st["cu_back"][1:].long())[seq]
    page, slot = st["pt"][seq, pos // PAGE].long(), pos % PAGE
    scale = pool[..., 4096:4104].contiguous().view(torch.float32)[page]
    out = []
    for which, place in enumerate(st["places"]):
        heads = torch.arange(hkv, device="cuda")[:, None]
        code = pool[page[:, None, None], heads, place[slot][:, None]].view(torch.float8_e4m3fn)
        out.append((code.float() * scale[..., which, None]).to(torch.bfloat16))
    return {"k": out[0], "v": out[1]}


def _plain_decode(st):
    """Softmax attention over the positions that each sequence's last token sees."""
    c, hkv = st["case"], st["case"]["kv_heads"]
    b, g = c["batch"], c["heads"] // hkv
    lens = st["seq_lens"].long()
    first = (lens - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(lens)
    lead = torch.minimum(first, torch.full_like(first, c["sinks"]))       # sinks before the window
    most = max(_sees(c, x - 1) for x in st["lens"])
    j = torch.arange(most, device="cuda")[None]
    pos = torch.where(j < lead[:, None], j, j + (first - lead)[:, None])
    seen = pos < lens[:, None]
    pos = torch.where(seen, pos, torch.zeros_like(pos))
    page, slot = st["pt"].gather(1, pos // PAGE).long(), pos % PAGE
    pool = st["pool"].view(st["pages"], hkv, REC)
    scale = pool[..., 4096:4104].contiguous().view(torch.float32)[page]      # [b, most, hkv, 2]
    heads = torch.arange(hkv, device="cuda")[:, None]

    def entries(which):
        code = pool[page[..., None, None], heads, st["places"][which][slot][:, :, None]]
        x = code.view(torch.float8_e4m3fn).float() * scale[..., which, None]
        return x.permute(0, 2, 1, 3)                                         # [b, hkv, most, D]

    q = st["q"].float().view(b, hkv, g, D)
    s = torch.matmul(q, entries(0).transpose(2, 3)) / math.sqrt(D)
    s.masked_fill_(~seen[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return (torch.matmul(p, entries(1)) / p.sum(-1, keepdim=True)).view(b, c["heads"], D)


def _sequence(st, b, dtype):
    """Keys and values [kv_heads, length, D] of sequence b."""
    n = st["lens"][b]
    ids = st["pt"][b, :(n + PAGE - 1) // PAGE].long()
    return [x.permute(1, 0, 2, 3).reshape(st["case"]["kv_heads"], -1, D)[:, :n]
            for x in _entries(st, ids, dtype)]


def _plain_prefill(st):
    c, hkv = st["case"], st["case"]["kv_heads"]
    g = c["heads"] // hkv
    out = torch.empty(c["n"], c["heads"], D, dtype=torch.bfloat16, device="cuda")
    at = 0
    for b, (n, length) in enumerate(zip(st["new"], st["lens"])):
        k, v = _sequence(st, b, torch.float32)
        q = st["q"][at:at + n].float().view(n, hkv, g, D).permute(1, 2, 0, 3).reshape(hkv, g * n, D)
        s = torch.matmul(q, k.transpose(1, 2)).view(hkv, g, n, length)
        s *= 1.0 / math.sqrt(D)
        row = torch.arange(length - n, length, device="cuda")[:, None]
        col = torch.arange(length, device="cuda")
        hidden = col > row
        if c["window"]:
            hidden |= (col <= row - c["window"]) & (col >= c["sinks"])
        s.masked_fill_(hidden, -math.inf)
        s = s.sub_(s.amax(-1, keepdim=True)).exp_()
        total = s.sum(-1, keepdim=True)
        o = torch.matmul(s.view(hkv, g * n, length), v).view(hkv, g, n, D) / total
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, c["heads"], D).to(torch.bfloat16)
        at += n
    return out


def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        if op == "norm":
            return _plain_norm(st)
        if op == "store":
            return _plain_store(st)
        return _plain_decode(st) if op == "decode" else _plain_prefill(st)
    from rotated_int2_kv_kvq_gb300 import kvq as K
    if op == "norm" and not c["back"]:
        K.kvq_norm_rope(st["h"], st["q"], st["k"], st["yq"], st["yk"], st["wq"], st["wk"], EPS,
                        st["positions"], st["rope"])
        return {"q": st["yq"], "k": st["yk"]}
    if op == "norm":
        K.kvq_norm_rope_backward(st["h"], st["q"], st["k"], st["dq"], st["dk"], st["yq"],
                                 st["yk"], st["wq"], st["wk"], st["dwq"], st["dwk"], EPS,
                                 st["positions"], st["rope"], st["ws"])
        return {"dq": st["yq"], "dk": st["yk"], "dwq": st["dwq"], "dwk": st["dwk"]}
    if op == "store":
        K.kvq_fp8_append(st["h"], st["pool"], st["pages"], st["k"], st["v"], st["cu"], st["pt"],
                         st["seq_lens"])
        K.kvq_fp8_read(st["h"], st["pool"], st["pages"], st["ko"], st["vo"], st["cu_back"],
                       st["pt"], st["seq_lens"])
        return {"k": st["ko"], "v": st["vo"]}
    if op == "decode":
        K.kvq_fp8_decode(st["h"], st["pool"], st["pages"], st["q"], st["pt"], st["seq_lens"],
                         st["out"], st["ws"], window=c["window"], sinks=c["sinks"])
        return st["out"]
    K.kvq_fp8_prefill(st["h"], st["pool"], st["pages"], st["q"], st["cu"], st["pt"],
                      st["seq_lens"], st["out"], st["ws"], window=c["window"], sinks=c["sinks"])
    return st["out"]


# ---- in 64 bits -----------------------------------------------------------------------------------

def _code_values():
    """The value of each of the 256 codes, from its bits; the two of all ones stand for NaN."""
    b = np.arange(256)
    ex, man = (b >> 3) & 15, b & 7
    v = np.where(ex == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (ex - 10.0)) * np.where(b > 127, -1, 1)
    v[[127, 255]] = np.nan
    return v


def _nearest_code(x):
    """x (|x| <= 448, float64) rounded to the nearest code's value, ties to the even mantissa."""
    up = torch.from_numpy(_code_values()[:127].copy()).cuda()      # 0 .. 448, ascending
    a = x.abs()
    hi = torch.searchsorted(up, a).clamp_(max=126)
    lo = (hi - 1).clamp_(min=0)
    to_lo, to_hi = a - up[lo], up[hi] - a
    take_lo = (to_lo < to_hi) | ((to_lo == to_hi) & (lo % 2 == 0))
    return torch.where(take_lo, up[lo], up[hi]) * torch.sign(x)


def _exact_store(st):
    """Page by page, head by head as the definition has it."""
    hkv, value = st["case"]["kv_heads"], torch.from_numpy(_code_values()).cuda()
    rec = st["pool"].view(st["pages"], hkv, REC)
    scale = rec[..., 4096:4104].contiguous().view(torch.float32).double()
    outs = ([], [])
    at = 0
    for b, (n, length, back) in enumerate(zip(st["new"], st["lens"], st["back"])):
        ids = st["pt"][b, :(length + PAGE - 1) // PAGE].long()
        start = length - n
        for which, x in enumerate((st["k"], st["v"])):
            held = value[rec[ids][..., st["places"][which]].long()]          # [pages, hkv, 16, D]
            s = scale[ids][..., which].clone()
            held = held * s[..., None, None]
            flat = held.permute(0, 2, 1, 3).reshape(-1, hkv, D).clone()
            first = start // PAGE
            fresh = first if start % PAGE == 0 else first + 1     # pages that this call begins
            if start % PAGE:
                flat[fresh * PAGE:] = 0
            else:
                flat[start:] = 0
            flat[start:length] = x[at:at + n].double()
            mark = torch.zeros(flat.shape[0], dtype=torch.bool, device="cuda")
            mark[start:length] = True
            top = (flat.abs().amax(-1) * mark[:, None]).view(-1, PAGE, hkv).amax(1)
            want = torch.where(top > 0, torch.ceil(torch.log2(top / 448.0)), -100.0).clamp_(min=-100)
            # log2 may be off by its last bit at a power of two: settle by the definition
            want = torch.where(top > 448.0 * 2.0 ** want, want + 1, want)
            want = torch.where((top <= 448.0 * 2.0 ** (want - 1)) & (want > -100), want - 1, want)
            touched = torch.arange(flat.shape[0] // PAGE, device="cuda") >= first
            grown = torch.maximum(2.0 ** want, s)
            grown[fresh:] = 2.0 ** want[fresh:]
            s = torch.where(touched[:, None], grown, s)
            unit = flat.view(-1, PAGE, hkv, D) / s[:, None, :, None]
            got = (_nearest_code(unit) * s[:, None, :, None]).view(-1, hkv, D)
            outs[which].append(got[length - back:length])
        at += n
    return {"k": torch.cat(outs[0]), "v": torch.cat(outs[1])}


def exact(case, seed):
    """From the definitions, in 64 bits: pairs turned as complex numbers, codes from a table of
    their values, attention one head at a time over all positions."""
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        rot, half, out = case["rot"], case["rot"] // 2, {}
        t = st["table"].double()[st["positions"].long()]
        turn = torch.complex(t[:, :half], t[:, half:])[:, None]
        a = slice(0, half) if case["style"] == "half" else slice(0, rot, 2)
        b = slice(half, rot) if case["style"] == "half" else slice(1, rot, 2)
        for name, w in (("q", st["wq"].double()), ("k", st["wk"].double())):
            x = st[name].double()
            size = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS)
            if not case["back"]:
                y = x / size * w
                z = torch.complex(y[..., a], y[..., b]) * turn
                y[..., a], y[..., b] = z.real, z.imag
                out[name] = y
                continue
            d = st["d" + name].double()
            z = torch.complex(d[..., a], d[..., b]) * turn.conj()
            d[..., a], d[..., b] = z.real, z.imag
            out["dw" + name] = torch.einsum("nhd,nhd->d", d, x / size)
            along = torch.einsum("nhd,nhd,d->nh", d, x, w)[..., None] / (D * size ** 3)
            out["d" + name] = d * w / size - x * along
        return out
    if op == "store":
        return _exact_store(st)
    hkv, g = case["kv_heads"], case["heads"] // case["kv_heads"]
    new = st["new"] if op == "prefill" else [1] * case["batch"]
    out = torch.empty(sum(new), case["heads"], D, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, length) in enumerate(zip(new, st["lens"])):
        keys, values = _sequence(st, b, torch.float64)
        row = torch.arange(length - n, length, device="cuda")[:, None]
        col = torch.arange(length, device="cuda")[None]
        seen = col <= row
        if case["window"]:
            seen &= (row - col < case["window"]) | (col < case["sinks"])
        for h in range(case["heads"]):
            s = st["q"][at:at + n, h].double() @ keys[h // g].T / math.sqrt(D)
            out[at:at + n, h] = torch.softmax(s.masked_fill(~seen, -math.inf), 1) @ values[h // g]
        at += n
    return out
