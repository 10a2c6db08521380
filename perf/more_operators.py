"""Attention over packed sequences with its gradients, and rotary positions with several axes: cases, plain forms and
exact values.

Three operators of a training step or of a prompt's pass:

* fwd: exact attention over sequences of different lengths that lie one after another in the rows of q, k and v (cu
  marks where each one's rows begin), grouped heads, causal or not, optionally with a sliding window.
* bwd: its gradients, from the forward's output and row statistics.
* rope: the rotation of queries and keys by positions with several axes (time, height, width), each pair of channels
  turned by the position on its own axis; its gradient is the rotation the other way round.
"""

import math
import random

import torch

own = False


# ------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one user's short prompt: nothing but latency
        _attn("fwd one short", "fwd", 1, 300, 12, 12, 64),
        # a server's prompts of very different lengths, grouped heads
        _attn("fwd prompts ragged", "fwd", 8, 4096, 32, 8, 128, ragged=7),
        # one long document: bound by the products
        _attn("fwd one long 16384", "fwd", 1, 16384, 32, 8, 128),
        # the patches of images of different sizes, each seeing all of its own, one key head per query head
        _attn("fwd images d64", "fwd", 24, 1369, 16, 16, 64, ragged=3, causal=False),
        # documents with a sliding window, groups of three, odd lengths
        _attn("fwd window d64", "fwd", 6, 5001, 12, 4, 64, ragged=11, window=700),
        # a gradient step on one short text
        _attn("bwd one short", "bwd", 1, 300, 12, 12, 64),
        # documents of different lengths packed into a training step, grouped heads
        _attn("bwd documents ragged", "bwd", 8, 4096, 32, 8, 128, ragged=7),
        # one long document, trained on
        _attn("bwd one long 8192", "bwd", 1, 8192, 16, 16, 128),
        # the patches of images again, small heads
        _attn("bwd images d64", "bwd", 24, 1369, 16, 16, 64, ragged=3, causal=False),
        # one token of a conversation with pictures in it
        _rope("rope one token", 1, 32, 8, 128, (16, 24, 24)),
        # a film's frames and the text around them
        _rope("rope film 32768", 32768, 32, 8, 128, (16, 24, 24)),
        # the gradient for patches of images: two axes, neighbours turned together, odd number of rows
        _rope("rope images back d64", 10007, 16, 16, 64, (16, 16), interleaved=True, inverse=True),
    ]


def _attn(name, op, B, L, Hq, Hkv, d, ragged=0, window=0, causal=True):
    return {"name": name, "op": op, "B": B, "L": L, "Hq": Hq, "Hkv": Hkv, "d": d, "ragged": ragged, "window": window,
            "causal": causal}


def _rope(name, T, Hq, Hkv, d, sections, interleaved=False, inverse=False):
    return {"name": name, "op": "rope", "T": T, "Hq": Hq, "Hkv": Hkv, "d": d, "sections": " ".join(map(str, sections)),
            "interleaved": interleaved, "inverse": inverse}


def _sections(c):
    """Pairs of channels on each axis."""
    return [int(n) for n in c["sections"].split()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    Hkv, G = rng.choice([(1, 8), (2, 4), (4, 3), (8, 4), (8, 8), (12, 1), (16, 1), (8, 5), (2, 7)])
    d = rng.choice([64, 128])
    if rng.random() < 0.25:
        pairs = rng.choice([d // 2, d // 2, d // 4])
        sections = rng.choice([(pairs,), (pairs // 2, pairs - pairs // 2), (pairs // 4, 3 * pairs // 8, 3 * pairs // 8),
                               (pairs // 4,) * 4, (pairs - 10, 5, 5)])
        return {"op": "rope", "T": _log(rng, 1, 32768 * 40 * 128 // (Hkv * (G + 1) * d) // 4), "Hq": Hkv * G, "Hkv": Hkv,
                "d": d, "sections": " ".join(map(str, sections)), "interleaved": rng.random() < 0.4, "inverse": rng.random() < 0.4}
    op = rng.choice(["fwd", "bwd"])
    B = _log(rng, 1, 64)
    # the plain form holds B x Hq x L x L scores, a few times over in the backward
    most = math.isqrt((1 << 32 if op == "fwd" else 1 << 30) // (B * Hkv * G))
    causal = rng.random() < 0.7
    return {"op": op, "B": B, "L": _log(rng, 1, min(most, 16384)), "Hq": Hkv * G, "Hkv": Hkv, "d": d,
            "ragged": rng.choice([0, rng.randrange(1, 1000)]), "causal": causal,
            "window": rng.choice([0, 0, _log(rng, 1, 4096)]) if causal else 0}


def _lens(c):
    """Each sequence's length: the case's own, or spread below it (an empty one among them now and then)."""
    if not c["ragged"]:
        return [c["L"]] * c["B"]
    rng = random.Random(c["ragged"])
    return [0 if c["B"] > 8 and rng.random() < 0.04 else rng.randint(1, c["L"]) for _ in range(c["B"])]


def work(c):
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    if c["op"] == "rope":
        T, rot = c["T"], 2 * sum(_sections(c))
        # queries and keys read and written; of the tables, a row's worth for each token; the positions
        return {"bytes": T * ((Hq + Hkv) * d * 2 * 2 + rot * 4 + 4 * len(_sections(c))), "flops": T * (Hq + Hkv) * rot * 3}
    lens = _lens(c)
    T, pairs = sum(lens), 0
    for n in lens:
        if not c["causal"]:
            pairs += n * n
        else:
            w = min(c["window"] or n, n)
            pairs += w * (w + 1) // 2 + (n - w) * w
    rows = T * d * 2
    stats = T * Hq * 4 + 4 * (len(lens) + 1)
    if c["op"] == "fwd":  # q, k, v read, o and lse written; two products
        return {"bytes": rows * (2 * Hq + 2 * Hkv) + stats, "flops": 4 * pairs * Hq * d}
    # q, o, do, k, v and lse read, dq, dk and dv written; five products
    return {"bytes": rows * (4 * Hq + 4 * Hkv) + stats, "flops": 10 * pairs * Hq * d}


# ------------------------------------------------------------------------------------------ the inputs
def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    s = {"case": c}
    if c["op"] == "rope":
        T, sections = c["T"], _sections(c)
        qk = torch.randn((T, (Hq + Hkv) * d), generator=g, device="cuda").to(torch.bfloat16)
        s["q"], s["k"] = qk[:, :Hq * d].view(T, Hq, d), qk[:, Hq * d:].view(T, Hkv, d)
        if len(sections) == 1:  # text: one axis
            s["positions"] = torch.arange(T, dtype=torch.int32, device="cuda")[None].contiguous()
        else:  # pictures: the last two axes walk over a grid, those before them count pictures
            i = torch.arange(T, device="cuda")
            h = w = max(1, math.isqrt(T) // 2)
            first = [i // (h * w) + 3 * a for a in range(len(sections) - 2)]
            grid = [i // w % h + i // (h * w), i % w + i // (h * w)]
            s["positions"] = torch.stack(first + grid).to(torch.int32)
        s["positions"] += 37  # what came before
        rot = 2 * sum(sections)
        inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        angle = torch.arange(int(s["positions"].max()) + 1, dtype=torch.float64, device="cuda")[:, None] * inv
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        return s
    lens = _lens(c)
    T, cu = sum(lens), [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s["T"], s["L"] = T, max(lens)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    # what the projection of a layer leaves: queries, keys and values of a token side by side
    qkv = torch.randn((T, (Hq + 2 * Hkv) * d), generator=g, device="cuda").to(torch.bfloat16)
    s["q"] = qkv[:, :Hq * d].view(T, Hq, d)
    s["k"] = qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
    s["v"] = qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d)
    if c["op"] == "bwd":
        s["o"], s["lse"] = _plain_fwd(s)
        s["do"] = torch.randn((T, Hq, d), generator=g, device="cuda").to(torch.bfloat16)
    if own:
        import exact_io_aware_33_gb300 as fa
        need = fa.fa_packed_fwd_workspace_bytes if c["op"] == "fwd" else fa.fa_packed_bwd_workspace_bytes
        s["workspace"] = torch.empty(need(c["B"], T, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------ the passes
def run(s):
    c = s["case"]
    if own:
        import exact_io_aware_33_gb300 as fa
        if c["op"] == "rope":
            q, k = fa.fa_rope_axes(s["q"], s["k"], s["positions"], (s["cos"], s["sin"]), sections=_sections(c),
                                   interleaved=c["interleaved"], inverse=c["inverse"])
            return {"q": q, "k": k}
        if c["op"] == "fwd":
            o, lse = fa.fa_packed_fwd(s["q"], s["k"], s["v"], s["cu"], causal=c["causal"], window=c["window"],
                                      workspace=s["workspace"])
            return {"o": o, "lse": lse}
        dq, dk, dv = fa.fa_packed_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["cu"], causal=c["causal"],
                                      window=c["window"], workspace=s["workspace"])
        return {"dq": dq, "dk": dk, "dv": dv}
    if c["op"] == "rope":
        q, k = _plain_rope(s, s["q"]), _plain_rope(s, s["k"])
        return {"q": q, "k": k}
    if c["op"] == "fwd":
        o, lse = _plain_fwd(s)
        return {"o": o, "lse": lse}
    dq, dk, dv = _plain_bwd(s)
    return {"dq": dq, "dk": dk, "dv": dv}


def _plain_rope(s, x):
    """x [T, H, d]; pair i of the turned channels takes the angle of the position on its own axis."""
    c = s["case"]
    sections = _sections(c)
    pairs = sum(sections)
    axis = torch.repeat_interleave(torch.arange(len(sections), device="cuda"), torch.tensor(sections, device="cuda"),
                                   output_size=pairs)
    at = s["positions"].long()[axis].t()                                  # [T, pairs]
    i = torch.arange(pairs, device="cuda")
    cos, sin = s["cos"][at, i][:, None], s["sin"][at, i][:, None]
    if c["inverse"]:
        sin = -sin
    y, rest = x[..., :2 * pairs].float(), x[..., 2 * pairs:].float()
    if c["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :pairs], y[..., pairs:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1).to(torch.bfloat16)


def _spread(s, x):
    """Packed rows [T, H, ...] in 32 bits, one sequence beside the other: [B, H, L, ...]; what is no row is 0."""
    i = torch.arange(s["L"], device="cuda")
    cu = s["cu"].long()
    rows = (cu[:-1, None] + i).clamp(max=s["T"] - 1)
    there = i < (cu[1:] - cu[:-1])[:, None]
    y = x[rows].float()
    return torch.where(there.view(there.shape + (1,) * (x.dim() - 1)), y, torch.zeros_like(y)).transpose(1, 2)


def _packed(s, x):
    """The other way round: [B, H, L, ...] to [T, H, ...]."""
    t = torch.arange(s["T"], device="cuda")
    cu = s["cu"].long()
    b = torch.searchsorted(cu, t, right=True) - 1
    return x[b, :, t - cu[b]]


def _masked_scores(s):
    """q k^T / sqrt(d) of each sequence's own pairs, -inf for the others: [B, Hkv, G, L, L]."""
    c, L = s["case"], s["L"]
    q = _spread(s, s["q"]).reshape(c["B"], c["Hkv"], -1, c["d"])          # the group's heads one under the other
    x = torch.matmul(q, _spread(s, s["k"]).transpose(2, 3)).mul_(1.0 / math.sqrt(c["d"]))
    x = x.view(c["B"], c["Hkv"], c["Hq"] // c["Hkv"], L, L)
    i = torch.arange(L, device="cuda")
    n = (s["cu"][1:] - s["cu"][:-1]).view(-1, 1, 1)
    far = i[:, None] - i
    seen = (i < n) & (i[:, None] < n)
    if c["causal"]:
        seen = seen & (far >= 0)
    if c["window"]:
        seen = seen & (far < c["window"])
    return x.masked_fill_(~seen[:, None, None], -math.inf)


def _plain_fwd(s):
    c, L = s["case"], s["L"]
    x = _masked_scores(s)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)       # rows behind a sequence
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(c["B"], c["Hkv"], -1, L), _spread(s, s["v"])).view(c["B"], c["Hq"], L, c["d"])
    total, top = total.view(c["B"], c["Hq"], L, 1), top.view(c["B"], c["Hq"], L, 1)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log())[..., 0]
    return _packed(s, o).to(torch.bfloat16), _packed(s, lse).contiguous()


def _plain_bwd(s):
    """P from the scores and lse, D = sum(do o); dv = P^T do, dS = P (do v^T - D), dq = scale dS k, dk = scale dS^T q."""
    c, L = s["case"], s["L"]
    B, Hkv, d, scale = c["B"], c["Hkv"], c["d"], 1.0 / math.sqrt(c["d"])
    lse, do = _spread(s, s["lse"]), _spread(s, s["do"])
    p = _masked_scores(s).sub_(lse.reshape(B, Hkv, -1, L, 1)).exp_().reshape(B, Hkv, -1, L)
    D = (do * _spread(s, s["o"])).sum(-1).reshape(B, Hkv, -1, 1)
    do = do.reshape(B, Hkv, -1, d)
    dv = torch.matmul(p.transpose(2, 3), do)
    p.mul_(torch.matmul(do, _spread(s, s["v"]).transpose(2, 3)).sub_(D))
    dq = torch.matmul(p, _spread(s, s["k"])).mul_(scale).view(B, c["Hq"], L, d)
    dk = torch.matmul(p.transpose(2, 3), _spread(s, s["q"]).reshape(B, Hkv, -1, d)).mul_(scale)
    return tuple(_packed(s, x).to(torch.bfloat16) for x in (dq, dk, dv))


# ------------------------------------------------------------------------------------------ 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        sections = _sections(c)
        pairs = sum(sections)
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
        pos = s["positions"].long()
        out = {}
        for name in ("q", "k"):
            y = s[name].double()
            for i in range(pairs):  # a pair of channels as one complex number, times e^(+-i angle)
                j = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + pairs)
                w = torch.complex(s["cos"][pos[axis[i]], i].double(), s["sin"][pos[axis[i]], i].double())[:, None]
                z = torch.complex(y[..., j[0]].contiguous(), y[..., j[1]].contiguous()) * (w.conj() if c["inverse"] else w)
                y[..., j[0]], y[..., j[1]] = z.real, z.imag
            out[name] = y
        return out
    lens = _lens(c)
    if sum(n * n for n in lens) * c["Hq"] * c["d"] * (4 if c["op"] == "fwd" else 10) > 5e12:
        return None
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    G, at, parts = Hq // Hkv, 0, []
    for n in lens:
        if n == 0:
            continue
        q, k, v = (s[m][at:at + n].double().transpose(0, 1) for m in ("q", "k", "v"))     # [heads, n, d]
        j = torch.arange(n, device="cuda")
        dk, dv = torch.zeros_like(k), torch.zeros_like(v)
        for i in range(0, n, 512):
            far = j[i:i + 512, None] - j
            off = ((far < 0) if c["causal"] else torch.zeros_like(far, dtype=torch.bool)) | (far >= (c["window"] or n + 1))
            here = slice(at + i, min(at + i + 512, at + n))
            qi = q[:, i:i + 512].reshape(Hkv, G, -1, d)
            x = torch.einsum("hgid,hjd->hgij", qi, k) / math.sqrt(d)
            if c["op"] == "fwd":
                x = x.masked_fill(off, -math.inf)
                z = torch.logsumexp(x, -1, keepdim=True)
                parts.append((torch.einsum("hgij,hjd->ihgd", (x - z).exp(), v).reshape(-1, Hq, d),
                              z[..., 0].permute(2, 0, 1).reshape(-1, Hq)))
                continue
            lse, do, o = (s[m][here].double().transpose(0, 1) for m in ("lse", "do", "o"))
            p = (x - lse.reshape(Hkv, G, -1, 1)).masked_fill(off, -math.inf).exp()
            do, o = do.reshape(Hkv, G, -1, d), o.reshape(Hkv, G, -1, d)
            dv += torch.einsum("hgij,hgid->hjd", p, do)
            ds = p * (torch.einsum("hgid,hjd->hgij", do, v) - (do * o).sum(-1, keepdim=True)) / math.sqrt(d)
            dk += torch.einsum("hgij,hgid->hjd", ds, qi)
            parts.append((torch.einsum("hgij,hjd->ihgd", ds, k).reshape(-1, Hq, d),))
        if c["op"] == "bwd":
            parts.append((dk.transpose(0, 1), dv.transpose(0, 1)))
        at += n
    if c["op"] == "fwd":
        return {"o": torch.cat([x[0] for x in parts]), "lse": torch.cat([x[1] for x in parts])}
    return {"dq": torch.cat([x[0] for x in parts if len(x) == 1]), "dk": torch.cat([x[0] for x in parts if len(x) == 2]),
            "dv": torch.cat([x[1] for x in parts if len(x) == 2])}
