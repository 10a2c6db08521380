"""The paged 8-bit key/value cache and the attention that reads it: cases, plain forms and exact values.

Two operators of a serving step:

* append: new keys and values (and, with them, the queries) are rotated by their positions; the rotated
  keys and the values are written to the pages of their sequences in e4m3, with one power-of-two scale
  per page and head for keys and one for values. A page that already holds tokens keeps its scale unless
  the new tokens need a larger one; then its older codes are rounded once more, to the larger scale.
* attn: queries over the cached keys and values of their own sequence, causal (the queries of a sequence
  are its last positions), optionally with a sliding window, grouped heads.

A batch is packed: the tokens of all sequences lie one after another in rows, cu_q marks where each
sequence's rows begin, kv_lens holds each sequence's length with its new tokens, and block_table names the
pages of each sequence.
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one user typing: a short conversation, one new token; nothing but latency
        _attn("attn one short", 1, 1, 300, 32, 8, 128, 16),
        # the decode workload of this repository's benchmark profile (8 x 32 heads over 8192 keys), paged
        _attn("attn decode b8 h32 8192", 8, 1, 8192, 32, 32, 128, 64),
        # a server's batch of requests of very different lengths, grouped heads
        _attn("attn decode b64 ragged", 64, 1, 16384, 32, 8, 128, 32, ragged=7),
        # one long document, one new token: few rows over a long axis, an odd length
        _attn("attn decode one long", 1, 1, 131071, 64, 8, 128, 128),
        # drafted tokens verified together, small heads, groups of three, small pages
        _attn("attn verify q5 d64", 24, 5, 4096, 12, 4, 64, 16, ragged=11),
        # a chunk of a long prompt over what is cached already: bound by the products
        _attn("attn chunk 2048 of 8192", 2, 2048, 8192, 32, 8, 128, 64),
        # fresh prompts of mixed lengths with a sliding window, one key head per query head
        _attn("attn prompts window d64", 8, 2048, 2048, 12, 12, 64, 64, ragged=5, window=700, fresh=True),
        # one user typing: one token rotated and written
        _append("append one", 1, 1, 301, 32, 8, 128, 16),
        # one token for each of a server's requests
        _append("append b256", 256, 1, 2048, 32, 8, 128, 64, ragged=3),
        # a whole prompt written at once
        _append("append prompt 8192", 1, 8192, 8192, 32, 8, 128, 64, fresh=True),
        # chunks of several prompts, small heads, half of each head rotated, in pairs of neighbours
        _append("append chunks d64", 16, 700, 2000, 12, 12, 64, 16, ragged=13, rot=32, interleaved=True),
    ]


def _attn(name, B, q, kv, Hq, Hkv, d, page, ragged=0, window=0, fresh=False):
    return {"name": name, "op": "attn", "B": B, "q": q, "kv": kv, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page,
            "ragged": ragged, "window": window, "fresh": fresh}


def _append(name, B, q, kv, Hq, Hkv, d, page, ragged=0, rot=0, interleaved=False, fresh=False):
    return {"name": name, "op": "append", "B": B, "q": q, "kv": kv, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page,
            "ragged": ragged, "rot": rot or d, "interleaved": interleaved, "fresh": fresh}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    Hkv, G = rng.choice([(1, 8), (2, 4), (4, 3), (8, 4), (8, 8), (12, 1), (32, 1), (8, 5)])
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    shape = rng.choice(["decode", "decode", "verify", "chunk", "prompt"])
    ragged = rng.choice([0, rng.randrange(1, 1000)])
    if shape == "decode":
        B = _log(rng, 1, 256)
        q, kv = 1, _log(rng, 1, max(2, min(131072, (1 << 22) // (B * Hkv))))
    elif shape == "verify":
        B = _log(rng, 1, 64)
        q, kv = rng.randrange(2, 17), _log(rng, 32, max(64, min(32768, (1 << 21) // (B * Hkv))))
    elif shape == "chunk":
        B = _log(rng, 1, 8)
        q = _log(rng, 17, max(18, 2048 // B))
        kv = q + _log(rng, 1, 8192)
    else:
        B = _log(rng, 1, 16)
        q = _log(rng, 17, 8192 // B)
        kv = q
    c = {"B": B, "q": q, "kv": max(q, kv), "Hq": Hkv * G, "Hkv": Hkv, "d": d, "page": page, "ragged": ragged}
    if rng.random() < 0.6:
        return {"op": "attn", **c, "window": rng.choice([0, 0, _log(rng, 1, 4096)]), "fresh": shape == "prompt"}
    return {"op": "append", **c, "rot": rng.choice([d, d, d // 2]), "interleaved": rng.random() < 0.4,
            "fresh": shape == "prompt"}


def _lens(c):
    """New tokens and total length of each sequence: the case's own, or spread below them where it is ragged."""
    if not c["ragged"]:
        return [c["q"]] * c["B"], [c["kv"]] * c["B"]
    rng = random.Random(c["ragged"])
    new, total = [], []
    for _ in range(c["B"]):
        n = rng.randint(1, c["q"])
        new.append(n)
        total.append(n if c["fresh"] else rng.randint(n, max(n, c["kv"])))
    return new, total


def work(c):
    new, total = _lens(c)
    T, d, Hq, Hkv, page = sum(new), c["d"], c["Hq"], c["Hkv"], c["page"]
    tables = 4 * (2 * c["B"] + 1) + 4 * sum(-(-t // page) for t in total)
    if c["op"] == "append":
        touched = sum(-(-t // page) - (t - n) // page for n, t in zip(new, total))
        # k, v and q read, q written, codes written, both tables of angles, the scales of the pages touched
        moved = T * (2 * Hkv * d * 2 + 2 * Hq * d * 2 + 2 * Hkv * d + c["rot"] * 4) + touched * Hkv * 8
        return {"bytes": moved + tables, "flops": T * (Hq + Hkv) * c["rot"] * 3 + T * 2 * Hkv * d * 2}
    pairs = keys = 0
    for n, t in zip(new, total):
        w = c["window"] or t
        # query i sits at position t - n + i and sees min(position + 1, window) keys
        lo, hi = t - n + 1, t
        short = max(0, min(hi, w) - lo + 1)
        pairs += (lo + min(hi, w)) * short // 2 + (n - short) * w
        keys += min(t, n + w - 1)
    moved = T * Hq * d * 4 + T * Hq * 4 + keys * Hkv * 2 * d + (keys // page + len(new)) * Hkv * 8
    return {"bytes": moved + tables, "flops": 4 * pairs * Hq * d}


# ------------------------------------------------------------------------------------------ the inputs
def _scale_of(amax):
    """Smallest power of two s with amax / s <= 448; 1 where there is nothing but zeros."""
    m, e = torch.frexp(amax)
    e = (e - torch.where(m <= 0.875, 9, 8)).clamp(-126, 127)
    s = ((e + 127).to(torch.int32) << 23).view(torch.float32)
    return torch.where(amax > 0, s, torch.ones_like(s))


def _tables(max_pos, rot):
    """cos and sin of position x frequency, in 64 bits, rounded once."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return angle.cos().float(), angle.sin().float()


def prepare(c, seed):
    new, total = _lens(c)
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, Hq, Hkv, d, page = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
    per_seq = [-(-t // page) for t in total]
    max_pages = max(per_seq)
    pages = sum(per_seq) + 3
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    # pages in the order in which a pool hands them out, which is none; unused entries name no page
    first = torch.tensor([0] + per_seq, device="cuda").cumsum(0)[:-1, None]
    col = torch.arange(max_pages, device="cuda")[None]
    used = col < torch.tensor(per_seq, device="cuda")[:, None]
    table = torch.where(used, perm[(first + col).clamp(max=pages - 1)], torch.full_like(perm[:1], -1)).contiguous()
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = {"case": c, "T": cu[-1], "max_q": max(new), "max_kv": max(total), "table": table,
         "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"),
         "lens": torch.tensor(total, dtype=torch.int32, device="cuda")}
    for name in ("k", "v"):
        # each head has channels of its own size, as keys and values have; whole pages hold numbers, also
        # behind the last token of a sequence, where they are left over from others
        size = torch.rand((1, Hkv, 1, d), generator=g, device="cuda") * 1.5 + 0.25
        codes = torch.empty((pages, Hkv, page, d), dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty((pages, Hkv), dtype=torch.float32, device="cuda")
        step = max(1, (1 << 27) // (Hkv * page * d))
        for at in range(0, pages, step):
            x = torch.randn((min(step, pages - at), Hkv, page, d), generator=g, device="cuda") * size
            scales[at:at + step] = _scale_of(x.abs().amax((2, 3)))
            codes[at:at + step] = (x / scales[at:at + step, :, None, None]).to(torch.float8_e4m3fn)
        s[name + "_pages"], s[name + "_scales"] = codes, scales
    if c["op"] == "append":
        # what the projection of a layer leaves: queries, keys and values of a token side by side
        qkv = torch.randn((s["T"], (Hq + 2 * Hkv) * d), generator=g, device="cuda").to(torch.bfloat16)
        s["q"] = qkv[:, :Hq * d].view(s["T"], Hq, d)
        s["k"] = qkv[:, Hq * d:(Hq + Hkv) * d].view(s["T"], Hkv, d)
        s["v"] = qkv[:, (Hq + Hkv) * d:].view(s["T"], Hkv, d)
        s["cos"], s["sin"] = _tables(s["max_kv"] + 5, c["rot"])
    else:
        s["q"] = torch.randn((s["T"], Hq, d), generator=g, device="cuda").to(torch.bfloat16)
    if own:
        import exact_io_aware_33_gb300 as fa
        s["cache"] = fa.PagedCache(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
        decode = s["max_q"] == 1
        s["batch"] = fa.PagedBatch(s["table"], s["lens"], None if decode else s["cu"], max_q=s["max_q"],
                                   max_kv=s["max_kv"])
        if c["op"] == "attn":
            n = fa.fa_paged_attn_workspace_bytes(s["cache"], s["batch"], Hq)
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------ the passes
def run(s):
    c = s["case"]
    if own:
        import exact_io_aware_33_gb300 as fa
        if c["op"] == "append":
            q = fa.fa_paged_append(s["cache"], s["batch"], s["k"], s["v"], q=s["q"], rope=(s["cos"], s["sin"]),
                                   interleaved=c["interleaved"])
        else:
            o, lse = fa.fa_paged_attn(s["cache"], s["batch"], s["q"], window=c["window"],
                                      workspace=s["workspace"])
    elif c["op"] == "append":
        q = _plain_append(s)
    else:
        o, lse = _plain_attn(s)
    if c["op"] == "append":
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"], "k_scales": s["k_scales"],
                "v_scales": s["v_scales"]}
    return {"o": o, "lse": lse}


def _rows(s):
    """Sequence and position of each packed row."""
    t = torch.arange(s["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"], t, right=True) - 1
    return b, (s["lens"][b] - s["cu"][b + 1] + t).long()


def _plain_rotate(x, cos, sin, interleaved):
    """x [T, H, d]; cos, sin [T, 1, rot / 2]. The first rot channels turn in pairs, the others stay."""
    rot = 2 * cos.shape[-1]
    x, rest = x[..., :rot].float(), x[..., rot:].float()
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1)


def _plain_append(s):
    c = s["case"]
    page = c["page"]
    b, pos = _rows(s)
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    where, slot = s["table"][b, pos // page].long(), pos % page
    q = _plain_rotate(s["q"], cos, sin, c["interleaved"]).to(torch.bfloat16)
    k = _plain_rotate(s["k"], cos, sin, c["interleaved"])
    # the page that each sequence's new tokens begin in, and how much of it was in use
    old = s["lens"] - (s["cu"][1:] - s["cu"][:-1])
    held = (old % page).long()
    begun = s["table"].gather(1, (old // page).long()[:, None].clamp(max=s["table"].shape[1] - 1))[:, 0].long().clamp(min=0)
    for name, x in (("k", k), ("v", s["v"].float())):
        codes, scales = s[name + "_pages"], s[name + "_scales"]
        raw = codes.view(torch.uint8)
        most = torch.zeros_like(scales).scatter_reduce_(0, where[:, None].expand(-1, c["Hkv"]), x.abs().amax(-1), "amax")
        kept = torch.zeros_like(scales).index_put_((begun,), torch.where(held[:, None] > 0, scales[begun], 0.0))
        # a page that none of the new tokens falls in keeps the scale that it has
        hit = torch.zeros_like(scales[:, 0]).index_put_((where,), torch.ones_like(scales[0, 0]))[:, None] > 0
        now = torch.where(hit, torch.maximum(_scale_of(most), kept), scales)
        before = codes[begun].float()
        ratio = (scales[begun] / now[begun])[:, :, None, None]
        stays = (torch.arange(page, device="cuda")[None] < held[:, None])[:, None, :, None]
        again = torch.where(stays, before * ratio, before).to(torch.float8_e4m3fn)
        raw[begun] = again.view(torch.uint8)
        new = (x / now[where][:, :, None]).to(torch.float8_e4m3fn)
        raw[where, :, slot] = new.view(torch.uint8)
        scales.copy_(now)
    return q


def _plain_attn(s):
    c = s["case"]
    B, Hq, Hkv, d, page, Q, L = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"], s["max_q"], s["max_kv"]
    G = Hq // Hkv
    at = s["table"].long().clamp(min=0)

    def values(codes, scales):  # [B, Hkv, L, d]
        x = codes[at].float() * scales[at][..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, -1, d)[:, :, :L]

    n = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(Q, device="cuda")
    rows = (s["cu"][:-1, None] + i).clamp(max=s["T"] - 1).long()
    q = s["q"][rows].float().view(B, Q, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, d)
    scores = torch.matmul(q, values(s["k_pages"], s["k_scales"]).transpose(2, 3)) * (1.0 / math.sqrt(d))
    j = torch.arange(L, device="cuda")
    p = (s["lens"] - n)[:, None] + i
    seen = (j <= p[..., None]) & (j < s["lens"][:, None, None])
    if c["window"]:
        seen = seen & (j > p[..., None] - c["window"])
    scores = scores.view(B, Hkv, Q, G, L).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    o = torch.matmul(weights.view(B, Hkv, Q * G, L), values(s["v_pages"], s["v_scales"])).view(B, Hkv, Q, G, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log())[..., 0]
    b, pos = _rows(s)
    row = pos - (s["lens"] - n)[b]
    return o[b, :, row].reshape(s["T"], Hq, d).to(torch.bfloat16), lse[b, :, row].reshape(s["T"], Hq)


# ------------------------------------------------------------------------------------------ 64 bits
def _e4m3_values():
    """The value of each of the 256 codes: sign, four bits of exponent (bias 7), three of fraction."""
    v = []
    for x in range(256):
        e, f = (x >> 3) & 15, x & 7
        a = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v.append((math.nan if x & 127 == 127 else a) * (-1 if x & 128 else 1))
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _power(e):
    """2 ** e in 64 bits, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest_e4m3(x):
    """x in 64 bits, |x| <= 448, to the nearest e4m3 value, halves to even."""
    _, e = torch.frexp(x)
    step = _power((e - 4).clamp(min=-9))
    return torch.round(x / step) * step


def exact(c, seed):
    s = prepare(c, seed)
    value = _e4m3_values()
    K, V = (s[n + "_pages"].view(torch.uint8) for n in ("k", "v"))
    Ks, Vs = s["k_scales"].double(), s["v_scales"].double()
    cu, lens, table, page, d = s["cu"].tolist(), s["lens"].tolist(), s["table"].long(), c["page"], c["d"]
    if c["op"] == "attn":
        G, o, lse = c["Hq"] // c["Hkv"], [], []
        for b, L in enumerate(lens):
            ids = table[b, :-(-L // page)]
            k = (value[K[ids].int()] * Ks[ids][..., None, None]).transpose(0, 1).flatten(1, 2)[:, :L]
            v = (value[V[ids].int()] * Vs[ids][..., None, None]).transpose(0, 1).flatten(1, 2)[:, :L]
            n = cu[b + 1] - cu[b]
            for i in range(0, n, 256):
                q = s["q"][cu[b] + i:min(cu[b] + i + 256, cu[b + 1])].double()
                m = q.shape[0]
                x = torch.einsum("mhgd,hld->hgml", q.view(m, c["Hkv"], G, d), k) / math.sqrt(d)
                far = (L - n + i + torch.arange(m, device="cuda"))[:, None] - torch.arange(L, device="cuda")
                x = x.masked_fill((far < 0) | (far >= (c["window"] or L + 1)), -math.inf)
                z = torch.logsumexp(x, -1, keepdim=True)
                o.append(torch.einsum("hgml,hld->mhgd", (x - z).exp(), v).reshape(m, c["Hq"], d))
                lse.append(z[..., 0].permute(2, 0, 1).reshape(m, c["Hq"]))
        return {"o": torch.cat(o), "lse": torch.cat(lse)}
    if max(s["max_q"], 1) * c["B"] > 40000:
        return None
    rot, cos, sin = c["rot"], s["cos"].double(), s["sin"].double()

    def turn(x, pos):  # [n, H, d]: each pair of channels as one complex number, times cos + i sin
        h, w = rot // 2, torch.complex(cos[pos], sin[pos])[:, None]
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :h], x[..., h:rot])
        z = torch.complex(a.contiguous(), b.contiguous()) * w
        y = x.clone()
        if c["interleaved"]:
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            y[..., :h], y[..., h:rot] = z.real, z.imag
        return y

    held = {"k": value[K.int()], "v": value[V.int()]}
    scales = {"k": Ks.clone(), "v": Vs.clone()}
    out_q = []
    for b, L in enumerate(lens):
        n = cu[b + 1] - cu[b]
        old, pos = L - n, torch.arange(L - n, L, device="cuda")
        out_q.append(turn(s["q"][cu[b]:cu[b + 1]].double(), pos))
        for name in ("k", "v"):
            x = s[name][cu[b]:cu[b + 1]].double()
            x = turn(x, pos) if name == "k" else x
            first = old // page
            count = -(-L // page) - first
            ids = table[b, first:first + count]
            # the sequence's pages side by side, from the first one touched: [H, count * page, d]
            lead = old - first * page
            wide = torch.zeros((c["Hkv"], count * page, d), dtype=torch.float64, device="cuda")
            wide[:, lead:lead + n] = x.transpose(0, 1)
            tile = wide.view(c["Hkv"], count, page, d).transpose(0, 1)
            amax = tile.abs().amax((2, 3))
            share = torch.where(amax > 0, amax, torch.full_like(amax, E4M3_MAX)) / E4M3_MAX
            m, e = torch.frexp(share)
            unit = _power(torch.where(m == 0.5, e - 1, e))
            if lead:
                unit[0] = torch.maximum(unit[0], scales[name][ids[0]])
            was = held[name][ids] * scales[name][ids][..., None, None]
            at = torch.arange(count * page, device="cuda").view(count, 1, page, 1)
            fresh = (at >= lead) & (at < lead + n)
            mine = at < lead + n
            codes = _nearest_e4m3(torch.where(fresh, tile, was) / unit[..., None, None])
            held[name][ids] = torch.where(mine, codes, held[name][ids])
            scales[name][ids] = unit
    return {"q": torch.cat(out_q), "k_pages": held["k"], "v_pages": held["v"], "k_scales": scales["k"],
            "v_scales": scales["v"]}
