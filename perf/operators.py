"""Work of the attention operators that stand between the qkv projection and the output projection.

Three operators, each in a plain form of elementary torch operations in 32 bits
(``own`` false) and as the call that a user makes of the library (``own`` true):

  norm_rope  RMS norm of every query and key head and the position rotation, bf16 in and out;
  append     the same on the way into a paged 8-bit cache: keys normalised, rotated and written
             with the values as E4M3 codes under one scale for each page and head (queries too);
  attn       causal attention of each sequence's newest tokens over that cache, optionally
             multiplied by the sigmoid of a gate.

Sizes.  The attention projections of the decode workloads are qkv N = 14336 and o_proj K = 6144:
24 query heads of 256 with a gate of the same size, 4 key and 4 value heads of 256
((24 + 24 + 4 + 4) * 256 = 14336, 24 * 256 = 6144), a quarter of each head rotated.  The others
(32 and 40 query heads of 128, 8 key heads) are generic.
"""
from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
MAX_EXP = 100  # a page's scale is a power of two in [2^-100, 2^100]


# ------------------------------------------------------------------- cases
def listed():
    gated = {"hq": 24, "hkv": 4, "d": 256, "rot": 64}
    plain = {"hq": 32, "hkv": 8, "d": 128, "rot": 128}
    return [
        # one decode token of one sequence: nothing but latency
        {"name": "norm_rope 1 token", "op": "norm_rope", "t": 1, "weights": True, "inter": False, **gated},
        # a whole prompt
        {"name": "norm_rope 8192 tokens", "op": "norm_rope", "t": 8192, "weights": True, "inter": False, **gated},
        # a decode step of 16 sequences: one token each, into pages that are partly full
        {"name": "append 16 x 1", "op": "append", "b": 16, "q": 1, "kv": 4099, "page": 64, "ragged": True,
         "weights": True, "inter": False, **gated},
        # seven prompts of different lengths, behind what their sequences hold already
        {"name": "append 7 ragged prompts", "op": "append", "b": 7, "q": 701, "kv": 1900, "page": 16, "ragged": True,
         "weights": False, "inter": True, **plain},
        # one long prompt into an empty cache
        {"name": "append 8192 tokens", "op": "append", "b": 1, "q": 8192, "kv": 8192, "page": 64, "ragged": False,
         "weights": True, "inter": False, **gated},
        # one token of one short conversation: nothing but latency
        {"name": "attn 1 x 301", "op": "attn", "b": 1, "q": 1, "kv": 301, "page": 16, "ragged": False, "gate": False,
         **plain},
        # the decode step that the projections' largest batch makes
        {"name": "attn 16 x 8191 gated", "op": "attn", "b": 16, "q": 1, "kv": 8191, "page": 64, "ragged": True,
         "gate": True, **gated},
        # a busy server: many sequences
        {"name": "attn 64 x 4096", "op": "attn", "b": 64, "q": 1, "kv": 4096, "page": 64, "ragged": True,
         "gate": False, **plain},
        # one very long document: all parallelism is along the cache
        {"name": "attn 1 x 131071", "op": "attn", "b": 1, "q": 1, "kv": 131071, "page": 64, "ragged": False,
         "gate": True, **gated},
        # speculative verification: five draft tokens a sequence
        {"name": "attn 8 x 5 over 16384", "op": "attn", "b": 8, "q": 5, "kv": 16384, "page": 64, "ragged": True,
         "gate": False, "hq": 40, "hkv": 8, "d": 128, "rot": 128},
        # a prompt into an empty cache
        {"name": "attn prompt 4096", "op": "attn", "b": 1, "q": 4096, "kv": 4096, "page": 32, "ragged": False,
         "gate": False, **plain},
        # one chunk of a long prompt, over what the earlier chunks left
        {"name": "attn chunk 2048 over 16384", "op": "attn", "b": 1, "q": 2048, "kv": 16384, "page": 64,
         "ragged": False, "gate": True, **gated},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 96, 128, 128, 256, 256])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 5, 6, 7, 8])
    rot = rng.choice([d, d // 2, d // 4])
    heads = {"hq": hkv * g, "hkv": hkv, "d": d, "rot": rot}
    op = rng.choice(["norm_rope", "append", "attn", "attn", "attn"])
    if op == "norm_rope":
        most = 8192 * 28 * 256 // ((hkv + hkv * g) * d)
        return {"op": op, "t": _log(rng, 1, min(most, 16384)), "weights": rng.random() < 0.7,
                "inter": rng.random() < 0.5, **heads}
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        b = _log(rng, 1, 64)
        most = max(1, 8192 * 32 * 256 // ((2 * hkv + hkv * g) * d * b))
        q = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, min(most, 8192)))
        kv = q + (0 if rng.random() < 0.3 else _log(rng, 1, max(1, 16384 // b)))
        return {"op": op, "b": b, "q": q, "kv": kv, "page": page, "ragged": rng.random() < 0.5,
                "weights": rng.random() < 0.7, "inter": rng.random() < 0.5, **heads}
    form = rng.choice(["decode", "decode", "verify", "prompt"])
    if form == "prompt":
        b = rng.choice([1, 1, 2, 3])
        q = _log(rng, 32, 4096 // b)
        past = 0 if rng.random() < 0.4 else _log(rng, 1, 8192)
        most = 2048 * 15360 * 24 * 256  # the largest listed chunk's pairs of positions, times heads and width
        past = min(past, max(0, most // (b * q * hkv * g * d) - q))
        kv = q + past
    else:
        b = _log(rng, 1, 96)
        q = 1 if form == "decode" else rng.randint(2, 8)
        kv = _log(rng, max(q, 16), max(q + 16, min(131072, 131071 * 4 * 256 // (b * hkv * d))))
    return {"op": "attn", "b": b, "q": q, "kv": kv, "page": page, "ragged": rng.random() < 0.5,
            "gate": rng.random() < 0.4, **heads}


def _lengths(c):
    """(new tokens, tokens with them) of every sequence: all alike, or between half of the most and the most."""
    b, q, kv, r = c["b"], c["q"], c["kv"], c["ragged"]
    step = [(i * 0.6180339887) % 1.0 * 0.5 if r else 0.0 for i in range(b)]
    qs = [max(1, q - int(q * s)) for s in step]
    return qs, [max(n, kv - int(kv * s)) for n, s in zip(qs, step)]


# ------------------------------------------------------------------ inputs
def _table(positions, rot):
    """cos and sin of every position and frequency: [positions][rot / 2 cos, rot / 2 sin], fp32."""
    half = rot // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    ang = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s, within 2^-100 .. 2^100 (2^-100 for amax = 0)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -MAX_EXP)).clamp(-MAX_EXP, MAX_EXP)
    return ((e.int() + 127) << 23).view(torch.float32)


def _paging(c, gen):
    """Page table (the pages of all sequences in a random order), cumulative new tokens and lengths."""
    qs, kvs = _lengths(c)
    need = [-(-n // c["page"]) for n in kvs]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    width = max(need)
    start = torch.tensor([sum(need[:i]) for i in range(c["b"])], device="cuda")
    at = (start[:, None] + torch.arange(width, device="cuda")).clamp(max=pages - 1)
    held = torch.arange(width, device="cuda") < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(held, order[at], torch.zeros_like(order[at])).contiguous()
    cu = torch.tensor([sum(qs[:i]) for i in range(c["b"] + 1)], dtype=torch.int32, device="cuda")
    return {"pages": pages, "table": table, "cu": cu, "kv": torch.tensor(kvs, dtype=torch.int32, device="cuda"),
            "tokens": sum(qs), "max_q": max(qs), "max_kv": max(kvs)}


def _cache(pages, c, gen):
    """Codes and scales of a cache whose channels differ in size, as keys' do."""
    shape = (pages, c["hkv"], c["page"], c["d"])
    size = torch.exp(torch.randn((c["hkv"], 1, c["d"]), generator=gen, device="cuda") * 0.4)
    x = torch.randn(shape, generator=gen, device="cuda") * size
    s = _pow2_scale(x.abs().amax((2, 3)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def _weight(c, gen):
    return (1.0 + 0.2 * torch.randn(c["d"], generator=gen, device="cuda")).bfloat16()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c)
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if c["op"] == "norm_rope":
        # q and k are slices of the projection's output rows
        row = torch.randn((c["t"], (hq + 2 * hkv) * d), generator=gen, device="cuda").bfloat16()
        first = torch.randint(0, 1024, (1,), generator=gen, device="cuda", dtype=torch.int32)
        s.update(q=row[:, :hq * d].unflatten(1, (hq, d)), k=row[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                 positions=first + torch.arange(c["t"], device="cuda", dtype=torch.int32),
                 table=_table(c["t"] + 1024, c["rot"]),
                 qw=_weight(c, gen) if c["weights"] else None, kw=_weight(c, gen) if c["weights"] else None)
        return s
    p = _paging(c, gen)
    kc, ks = _cache(p["pages"], c, gen)
    vc, vs = _cache(p["pages"], c, gen)
    s.update(p, kc=kc, ks=ks, vc=vc, vs=vs)
    if c["op"] == "append":
        row = torch.randn((p["tokens"], (hq + 2 * hkv) * d), generator=gen, device="cuda").bfloat16()
        heads = row.unflatten(1, (hq + 2 * hkv, d))
        s.update(q=heads[:, :hq], k=heads[:, hq:hq + hkv], v=heads[:, hq + hkv:],
                 rope=_table(p["max_kv"], c["rot"]),
                 qw=_weight(c, gen) if c["weights"] else None, kw=_weight(c, gen) if c["weights"] else None)
        return s
    s["q"] = (1.5 * torch.randn((p["tokens"], hq, d), generator=gen, device="cuda")).bfloat16()
    s["gate"] = torch.randn((p["tokens"], hq, d), generator=gen, device="cuda").bfloat16() if c["gate"] else None
    return s


# ------------------------------------------------------------- plain forms
def _norm(x, w):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotate(x, cs, rot, inter):
    """x [T, H, D] with its first `rot` entries rotated by the rows cs [T, rot] of the table."""
    half = rot // 2
    cos, sin = cs[:, None, :half], cs[:, None, half:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :half], x[..., half:rot])
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if inter else torch.cat(y, -1)
    return torch.cat([y, x[..., rot:]], -1)


def _norm_rope(s):
    cs = s["table"][s["positions"].long()]
    q = _rotate(_norm(s["q"], s["qw"]), cs, s["rot"], s["inter"])
    k = _rotate(_norm(s["k"], s["kw"]), cs, s["rot"], s["inter"])
    return q.bfloat16(), k.bfloat16()


def _token_places(s):
    """Sequence and position of every new token."""
    t = torch.arange(s["tokens"], device="cuda")
    seq = (t[:, None] >= s["cu"][None, 1:]).sum(1)
    return seq, t - s["cu"][1:].long()[seq] + s["kv"].long()[seq]


def _store(codes, scales, x, page, slot, first_slot):
    """Writes x [T, H, D] at (page, slot): every page's scale grows to what its new tokens need."""
    amax = torch.zeros_like(scales).index_reduce(0, page, x.abs().amax(-1), "amax")
    touched = torch.zeros(scales.shape[0], device="cuda", dtype=torch.bool)
    touched[page] = True
    at = touched.nonzero()[:, 0]
    kept = torch.zeros(scales.shape[0], device="cuda", dtype=torch.long)
    kept[page] = first_slot  # tokens that the page held before this call
    kept, old = kept[at], scales[at]
    new = torch.where(kept[:, None] > 0, torch.maximum(old, _pow2_scale(amax[at])), _pow2_scale(amax[at]))
    held = codes[at]
    again = (held.float() * (old / new)[:, :, None, None]).to(torch.float8_e4m3fn)
    is_old = (torch.arange(codes.shape[2], device="cuda") < kept[:, None])[:, None, :, None]
    codes[at] = torch.where(is_old, again.view(torch.uint8), held.view(torch.uint8)).view(torch.float8_e4m3fn)
    scales[at] = new
    codes[page, :, slot] = (x / scales[page][:, :, None]).to(torch.float8_e4m3fn)


def _append(s):
    seq, pos = _token_places(s)
    cs = s["rope"][pos]
    q = _rotate(_norm(s["q"], s["qw"]), cs, s["rot"], s["inter"])
    k = _rotate(_norm(s["k"], s["kw"]), cs, s["rot"], s["inter"])
    page = s["table"][seq, pos // s["page"]].long()
    slot = pos % s["page"]
    begin = (s["kv"] - (s["cu"][1:] - s["cu"][:-1])).long()[seq]  # position of the sequence's first new token
    first_slot = torch.where(begin // s["page"] == pos // s["page"], begin % s["page"], torch.zeros_like(begin))
    _store(s["kc"], s["ks"], k, page, slot, first_slot)
    _store(s["vc"], s["vs"], s["v"].float(), page, slot, first_slot)
    return q.bfloat16(), s["kc"], s["ks"], s["vc"], s["vs"]


def _gather(codes, scales, table):
    """The table's pages as fp32 [B, H, L, D]."""
    x = codes[table.long()].float() * scales[table.long()][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _attn(s):
    b, hq, hkv, d = s["b"], s["hq"], s["hkv"], s["d"]
    seq, pos = _token_places(s)
    i = torch.arange(s["tokens"], device="cuda") - s["cu"].long()[seq]
    q = torch.zeros((b, s["max_q"], hq, d), device="cuda")
    q[seq, i] = s["q"].float()
    q = q.view(b, s["max_q"], hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hkv, G Q, D]
    k, v = _gather(s["kc"], s["ks"], s["table"]), _gather(s["vc"], s["vs"], s["table"])
    at = torch.full((b, s["max_q"]), -1, device="cuda", dtype=torch.long)
    at[seq, i] = pos
    seen = torch.arange(k.shape[2], device="cuda") <= at[:, :, None]  # [B, Q, L]
    x = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    x = x.view(b, hkv, hq // hkv, s["max_q"], -1).masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = x.sum(-1, keepdim=True)
    x = x / torch.where(total > 0, total, torch.ones_like(total))
    y = (x.flatten(2, 3) @ v).view(b, hkv, hq // hkv, s["max_q"], d).permute(0, 3, 1, 2, 4)[seq, i].flatten(1, 2)
    if s["gate"] is not None:
        y = y / (1.0 + torch.exp(-s["gate"].float()))
    return y.bfloat16()


# --------------------------------------------------------------------- run
def run(state):
    s = state
    if not own:
        return {"norm_rope": _norm_rope, "append": _append, "attn": _attn}[s["op"]](s)
    import nvfp4_weight_quantized_gemv_gb300 as nv
    if s["op"] == "norm_rope":
        return nv.nvfp4_qk_norm_rope(s["q"], s["k"], s["positions"], s["table"], q_weight=s["qw"], k_weight=s["kw"],
                                     eps=EPS, interleaved=s["inter"])
    if s["op"] == "append":
        q = nv.nvfp4_kv_append(s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["kv"],
                               s["max_q"], cos_sin=s["rope"], k_weight=s["kw"], q=s["q"], q_weight=s["qw"], eps=EPS,
                               interleaved=s["inter"])
        return q, s["kc"], s["ks"], s["vc"], s["vs"]
    return nv.nvfp4_attn_paged(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["kv"], s["max_q"],
                               s["max_kv"], gate=s["gate"])


def work(case):
    c = case
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if c["op"] == "norm_rope":
        n = c["t"] * (hq + hkv)
        return {"bytes": 4 * n * d + c["t"] * 4 * c["rot"], "flops": n * (4 * d + 3 * c["rot"])}
    qs, kvs = _lengths(c)
    t = sum(qs)
    if c["op"] == "append":  # rows in, q out, codes out, a scale for each touched page and head in and out, the table
        pages = sum(-(-kv // c["page"]) - (kv - q) // c["page"] for q, kv in zip(qs, kvs))
        return {"bytes": t * (4 * hq * d + 2 * 2 * hkv * d + 2 * hkv * d + 4 * c["rot"]) + pages * hkv * 2 * 8,
                "flops": t * (hq + hkv) * (4 * d + 3 * c["rot"]) + t * hkv * d * 4}
    pairs = sum(q * kv - q * (q - 1) // 2 for q, kv in zip(qs, kvs))
    pages = sum(-(-kv // c["page"]) for kv in kvs)
    return {"bytes": 2 * sum(kvs) * hkv * d + pages * hkv * 8 + t * hq * d * (6 if c["gate"] else 4),
            "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------- exact
def _exact_heads(x, w, cs, rot, inter):
    """Norm and rotation in 64 bits as a product of complex numbers."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    half = rot // 2
    turn = torch.complex(cs[:, :half].double(), cs[:, half:].double())[:, None]
    first = torch.arange(half, device="cuda") * 2 if inter else torch.arange(half, device="cuda")
    second = first + (1 if inter else half)
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_e4m3(x):
    """x rounded to the nearest E4M3 value, ties to even, in 64 bits."""
    _, e = torch.frexp(x)
    step = (((e - 4).clamp(min=-9).long() + 1023) << 52).view(torch.float64)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_scale(amax):
    e = -MAX_EXP
    while amax > E4M3_MAX * 2.0 ** e and e < MAX_EXP:
        e += 1
    return 2.0 ** e


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm_rope":
        cs = s["table"][s["positions"].long()]
        return (_exact_heads(s["q"], s["qw"], cs, c["rot"], c["inter"]),
                _exact_heads(s["k"], s["kw"], cs, c["rot"], c["inter"]))
    qs, kvs = _lengths(c)
    table = s["table"].tolist()
    if c["op"] == "append":
        pos = torch.cat([torch.arange(kv - q, kv, device="cuda") for q, kv in zip(qs, kvs)])
        cs = s["rope"][pos]
        new_k = _exact_heads(s["k"], s["kw"], cs, c["rot"], c["inter"])
        out = [_exact_heads(s["q"], s["qw"], cs, c["rot"], c["inter"])]
        for codes, scales, new in ((s["kc"], s["ks"], new_k), (s["vc"], s["vs"], s["v"].double())):
            codes, scales, at = codes.double(), scales.double(), 0
            for b, (q, kv) in enumerate(zip(qs, kvs)):
                p = kv - q
                while p < kv:
                    slot, n = p % c["page"], min(c["page"] - p % c["page"], kv - p)
                    part, page = new[at:at + n].transpose(0, 1), table[b][p // c["page"]]  # [H, n, D]
                    need = torch.tensor([_exact_scale(a) for a in part.abs().amax((1, 2)).tolist()], device="cuda",
                                        dtype=torch.float64)
                    if slot:
                        need = torch.maximum(need, scales[page])
                        codes[page, :, :slot] = _exact_e4m3(
                            codes[page, :, :slot] * (scales[page] / need)[:, None, None])
                    scales[page] = need
                    codes[page, :, slot:slot + n] = _exact_e4m3(part / need[:, None, None])
                    p, at = p + n, at + n
            out += [codes, scales]
        return tuple(out)
    g, y, at = c["hq"] // c["hkv"], [], 0
    for b, (q, kv) in enumerate(zip(qs, kvs)):
        pages = torch.tensor(table[b][:-(-kv // c["page"])], device="cuda")
        k, v = ((x[pages].double() * z[pages].double()[:, :, None, None]).transpose(0, 1).flatten(1, 2)[:, :kv]
                for x, z in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
        rows = torch.empty((q, c["hq"], c["d"]), device="cuda", dtype=torch.float64)
        hidden = torch.arange(kv, device="cuda") > torch.arange(kv - q, kv, device="cuda")[:, None]
        for h in range(c["hq"]):
            z = s["q"][at:at + q, h].double() @ k[h // g].T / math.sqrt(c["d"])
            rows[:, h] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v[h // g]
        y.append(rows)
        at += q
    y = torch.cat(y)
    return y if s["gate"] is None else y * torch.sigmoid(s["gate"].double())


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(8)]:
        print(case, work(case))
