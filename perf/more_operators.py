"""Work of the operators around a batch of requests over the paged cache.

Three operators, each in a plain form of elementary torch operations (``own`` false) and as the call
that a user makes of the library (``own`` true):

  tables  block tables, slot map, positions and cumulative lengths of a step, from the requests' lengths
          and a ring of free pages;
  shared  attention over the paged 8-bit cache for a batch whose sequences share long prefixes;
  verify  drafted tokens against the target's probabilities, from given random numbers.

Sizes.  Heads are those of the attention workloads: 24 query heads of 256 with 4 kv heads and gates, 32
and 40 query heads of 128 with 8 kv heads.  Vocabularies, batches and lengths are generic.
"""
from __future__ import annotations

import math
import random

import torch

own = False


# ------------------------------------------------------------------- cases
def listed():
    gated = {"hq": 24, "hkv": 4, "d": 256, "gate": True}
    plain = {"hq": 32, "hkv": 8, "d": 128, "gate": False}
    return [
        # the tables of a decode step of 16 requests: nothing but latency
        {"name": "tables 16 requests", "op": "tables", "b": 16, "mix": "decode", "q": 1, "kv": 4099, "page": 64},
        # a busy server: most requests bring five tokens, some a whole prompt, some have ended and give their pages back
        {"name": "tables 1024 mixed requests", "op": "tables", "b": 1024, "mix": "mixed", "q": 400, "kv": 3001, "page": 16},
        # four drafts of one request over a small vocabulary: nothing but latency
        {"name": "verify 1 x 4 of 32000", "op": "verify", "b": 1, "drafts": 4, "vocab": 32000, "given": True, "ragged": False},
        # drafts of no distribution (looked up in the text), an odd vocabulary
        {"name": "verify 16 x 8 of 100003, looked up", "op": "verify", "b": 16, "drafts": 8, "vocab": 100003, "given": False,
         "ragged": True},
        # a busy server with a draft model
        {"name": "verify 64 x 5 of 131072", "op": "verify", "b": 64, "drafts": 5, "vocab": 131072, "given": True,
         "ragged": True},
        # four samples of one prompt: few rows
        {"name": "shared 4 x 1 over 2048", "op": "shared", "groups": 1, "b": 4, "q": 1, "prefix": 2048, "own": 90, "page": 16,
         **plain},
        # a decode step of 16 requests behind one instruction text
        {"name": "shared 16 x 1 over 8192 gated", "op": "shared", "groups": 1, "b": 16, "q": 1, "prefix": 8192, "own": 509,
         "page": 64, **gated},
        # a busy server, everybody behind the same long text
        {"name": "shared 64 x 1 over 16384", "op": "shared", "groups": 1, "b": 64, "q": 1, "prefix": 16384, "own": 1021,
         "page": 64, **plain},
        # speculative verification: four drafts a request
        {"name": "shared 32 x 5 over 32768", "op": "shared", "groups": 1, "b": 32, "q": 5, "prefix": 32768, "own": 300,
         "page": 32, "hq": 40, "hkv": 8, "d": 128, "gate": False},
        # several texts of different lengths, eight requests each
        {"name": "shared 6 groups of 8 x 1 over 7000", "op": "shared", "groups": 6, "b": 48, "q": 1, "prefix": 7000, "own": 700,
         "page": 64, **gated},
        # questions about one document, a whole prompt each
        {"name": "shared 8 x 257 over 8192", "op": "shared", "groups": 1, "b": 8, "q": 257, "prefix": 8192, "own": 257,
         "page": 64, **plain},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "verify", "shared", "shared"])
    if op == "tables":
        mix = rng.choice(["decode", "mixed"])
        b = _log(rng, 1, 1024)
        return {"op": op, "b": b, "mix": mix, "q": rng.randint(1, 8) if mix == "decode" else _log(rng, 8, 400),
                "kv": _log(rng, 16, min(32768, 1024 * 3001 // b)), "page": rng.choice([16, 32, 64, 128])}
    if op == "verify":
        b, drafts = _log(rng, 1, 64), rng.randint(0, 8)
        most = 64 * 6 * 131072 // (b * (drafts + 1))
        return {"op": op, "b": b, "drafts": drafts, "vocab": _log(rng, 1000, min(160000, most)),
                "given": rng.random() < 0.6, "ragged": rng.random() < 0.5}
    d = rng.choice([64, 96, 128, 128, 256, 256])
    hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 6, 7, 8])
    groups = rng.choice([1, 1, 1, 2, 5])
    b = groups * _log(rng, 2, max(2, 64 // groups))
    form = rng.choice(["decode", "decode", "verify", "prompt"])
    q = {"decode": 1, "verify": rng.randint(2, 8), "prompt": _log(rng, 9, max(9, 2056 // b))}[form]
    # of the largest listed one: the pairs of positions, times heads and width, and the codes of all sequences
    most = 8 * 257 * 8449 * 32 * 128 // (b * q * hkv * g * d)
    own_most = min(most // 2, 64 * 1021 * 8 * 128 // (b * hkv * d), 4096)
    return {"op": op, "groups": groups, "b": b, "q": q, "prefix": _log(rng, 128, max(256, min(32768, most // 2))),
            "own": max(q, _log(rng, 1, max(2, own_most))), "page": rng.choice([16, 32, 64, 128]), "hq": hkv * g, "hkv": hkv,
            "d": d, "gate": rng.random() < 0.4}


# ------------------------------------------------------------------ inputs
def _spread(n):
    """Numbers in [0, 1) that differ for neighbours."""
    return [(i * 0.6180339887) % 1.0 for i in range(n)]


def _table_lengths(c):
    """(held, new) tokens of every request before the step; a mixed batch has prompts and requests that have ended."""
    kv = [max(1, c["kv"] - int(c["kv"] * s * 0.7)) for s in _spread(c["b"])]
    q = [c["q"]] * c["b"]
    if c["mix"] == "mixed":
        for i in range(c["b"]):
            if i % 16 == 5:  # a prompt, nothing held yet
                kv[i], q[i] = 0, max(1, c["q"] - (i % 64))
            elif i % 16 == 11:  # ended: all its pages are given back
                kv[i], q[i] = 0, 0
            else:
                q[i] = min(5, c["q"])
    return kv, q


def _table_held(c, kv):
    """Pages that every request holds; requests that have ended hold what their text took."""
    return [-(-(c["kv"] // 2 if c["mix"] == "mixed" and i % 16 == 11 else n) // c["page"]) for i, n in enumerate(kv)]


def _shared_lengths(c):
    """(prefix of every group, requests of every group, own tokens of every request); prefixes are whole pages."""
    g = c["groups"]
    prefix = [max(1, int(c["prefix"] * (1 - 0.5 * s)) // c["page"]) * c["page"] for s in _spread(g)]
    of = [c["b"] // g] * g
    return prefix, of, [max(c["q"], c["own"] - int(c["own"] * s * 0.5)) for s in _spread(c["b"])]


def _codes(pages, c, gen):
    """Codes and scales of a cache whose channels differ in size, as keys' do."""
    size = torch.exp(torch.randn((c["hkv"], 1, c["d"]), generator=gen, device="cuda") * 0.4)
    x = torch.randn((pages, c["hkv"], c["page"], c["d"]), generator=gen, device="cuda") * size
    s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _sums(values):
    out = [0]
    for v in values:
        out.append(out[-1] + v)
    return out


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c)
    if c["op"] == "tables":
        kv, q = _table_lengths(c)
        held = _table_held(c, kv)
        width = max(max(-(-(n + m) // c["page"]) for n, m in zip(kv, q)), max(held)) + 1
        grow = sum(max(0, -(-(n + m) // c["page"]) - h) for n, m, h in zip(kv, q, held))
        free = grow + 7
        ring = sum(held) + free
        order = torch.randperm(ring, generator=gen, device="cuda", dtype=torch.int32)
        first = _ints(_sums(held)[:-1], torch.int64)
        at = (first[:, None] + torch.arange(width, device="cuda")).clamp(max=ring - 1)
        has = torch.arange(width, device="cuda") < _ints(held)[:, None]
        head = torch.randint(0, 1 << 40, (1,), generator=gen, device="cuda")
        pages = torch.zeros(ring, dtype=torch.int32, device="cuda")
        pages[(head + torch.arange(free, device="cuda")) % ring] = order[sum(held):]
        s.update(table=torch.where(has, order[at], torch.zeros_like(order[at])).contiguous(), held=_ints(held), pages=pages,
                 span=torch.cat([head, head + free]), lens=_ints(kv), new=_ints(q), tokens=sum(q) + 3)
        return s
    if c["op"] == "verify":
        n = [max(0, c["drafts"] - int(c["drafts"] * f * 0.7)) if c["ragged"] else c["drafts"] for f in _spread(c["b"])]
        cu = _sums([k + 1 for k in n])
        x = 2.5 * torch.randn((cu[-1], c["vocab"]), generator=gen, device="cuda")
        target = torch.softmax(x, 1)
        if c["given"]:  # a draft model that is near the target
            x += 0.5 * torch.randn((cu[-1], c["vocab"]), generator=gen, device="cuda")
        drawn = torch.multinomial(torch.softmax(x, 1), 1, generator=gen)[:, 0].int()
        s.update(target=target, draft=torch.softmax(x, 1) if c["given"] else None, cu=_ints(cu),
                 tokens=torch.cat([drawn[-1:], drawn[:-1]]), u=torch.rand(cu[-1], generator=gen, device="cuda"),
                 pick=torch.rand(c["b"], generator=gen, device="cuda"),
                 lens=_ints([100 + 7 * i + k for i, k in enumerate(n)]))
        return s
    prefix, of, mine = _shared_lengths(c)
    group = [g for g, k in enumerate(of) for _ in range(k)]
    page = c["page"]
    pre, need = [p // page for p in prefix], [-(-n // page) for n in mine]
    pages = sum(pre) + sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    width = max(pre[g] + k for g, k in zip(group, need))
    table = torch.zeros((c["b"], width), dtype=torch.int32, device="cuda")
    pre0, own0 = _sums(pre), _sums(need)
    for b, (g, k) in enumerate(zip(group, need)):
        table[b, :pre[g]] = order[pre0[g]:pre0[g + 1]]
        table[b, pre[g]:pre[g] + k] = order[pre0[-1] + own0[b]:pre0[-1] + own0[b + 1]]
    kc, ks = _codes(pages, c, gen)
    vc, vs = _codes(pages, c, gen)
    tokens = c["b"] * c["q"]
    q = (1.5 * torch.randn((tokens, c["hq"], c["d"]), generator=gen, device="cuda")).bfloat16()
    s.update(table=table, kc=kc, ks=ks, vc=vc, vs=vs, queries=q,
             gates=torch.randn(q.shape, generator=gen, device="cuda").bfloat16() if c["gate"] else None,
             cu=_ints([c["q"] * i for i in range(c["b"] + 1)]), lens=_ints([prefix[g] + n for g, n in zip(group, mine)]),
             group_cu=_ints(_sums(of)), prefixes=_ints(prefix), prefix_list=prefix, of=of, max_own=max(mine),
             max_kv=max(prefix[g] + n for g, n in zip(group, mine)), max_group=max(of) * c["q"])
    return s


# ------------------------------------------------------------- plain forms
def _tables(s):
    table, held, page = s["table"], s["held"].long(), s["page"]
    kv, q = s["lens"].long(), s["new"].long()
    head, tail = s["span"][0], s["span"][1]
    ring, width = s["pages"].shape[0], table.shape[1]
    fits = (kv >= 0) & (q >= 0) & (kv + q <= width * page)
    fits &= (q == 0) | (torch.cumsum(torch.where(fits, q, 0), 0) <= s["tokens"])
    need = (kv + q + page - 1) // page
    grow = torch.where(fits, (need - held).clamp(min=0), 0)
    taken = torch.cumsum(grow, 0)
    fits &= (grow == 0) | (taken <= tail - head)
    grow = torch.where(fits, grow, 0)
    back = torch.where(fits, (held - need).clamp(min=0), 0)
    q = torch.where(fits, q, 0)
    cu = torch.cat([torch.zeros_like(q[:1]), torch.cumsum(q, 0)])
    # entries [held, held + grow) from the ring's head, entries [held - back, held) to its tail
    i = torch.arange(width, device="cuda")
    seq, at = ((i >= held[:, None]) & (i < (held + grow)[:, None])).nonzero(as_tuple=True)
    table[seq, at] = s["pages"][(head + (taken - grow)[seq] + at - held[seq]) % ring]
    seq, at = ((i >= (held - back)[:, None]) & (i < held[:, None])).nonzero(as_tuple=True)
    s["pages"][(tail + torch.arange(seq.shape[0], device="cuda")) % ring] = table[seq, at]
    t = torch.arange(s["tokens"], device="cuda")
    live = t < cu[-1]
    seq = (t[:, None] >= cu[None, 1:]).sum(1).clamp(max=q.shape[0] - 1)
    pos = torch.where(live, kv[seq] + t - cu[seq], 0)
    slot = torch.where(live, table[seq, pos // page].long() * page + pos % page, -1)
    span = torch.stack([head + grow.sum(), tail + back.sum()])
    return (cu.int(), (kv + q).int(), pos.int(), slot, (held + grow - back).int(), span, table, s["pages"])


def _verify(s):
    cu, b, v = s["cu"].long(), s["b"], s["vocab"]
    rows = s["tokens"].shape[0]
    t = torch.arange(rows, device="cuda")
    seq = (t[:, None] >= cu[None, 1:]).sum(1)
    drafted = t + 1 < cu[seq + 1]  # this row's distribution judges the next token
    x = s["tokens"].long()[(t + 1).clamp(max=rows - 1)]
    p = s["target"][t, x].double()
    q = s["draft"][t, x].double() if s["draft"] is not None else torch.ones_like(p)
    bad = drafted & ~(s["u"].double() * q < p)
    first = torch.full((b,), 1 << 30, device="cuda", dtype=torch.long).scatter_reduce(
        0, seq, torch.where(bad, t, torch.full_like(t, 1 << 30)), "amin")
    at = torch.minimum(first, cu[1:] - 1)  # the row that the new token is drawn from
    n = at - cu[:-1]
    p = s["target"][at].double()
    over = (at + 1 < cu[1:])[:, None]  # a draft was refused
    if s["draft"] is not None:
        r = torch.where(over, (p - s["draft"][at].double()).clamp(min=0), p)
    else:
        mine = torch.arange(v, device="cuda") == x[at][:, None]
        r = torch.where(over & mine, torch.zeros_like(p), p)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p)
    c = torch.cumsum(r, 1)
    last = torch.where(r > 0, torch.arange(v, device="cuda"), 0).amax(1)
    new = torch.minimum((c <= s["pick"].double()[:, None] * c[:, -1:]).sum(1), last)
    i = t - cu[seq]
    out = torch.where(i < n[seq], x, torch.where(i == n[seq], new[seq], -1))
    return out.int(), n.int(), new.int(), (s["lens"] - (cu[1:] - 1 - at)).int()


def _pages(codes, scales, table):
    """The table's pages as fp32 [.., H, L, D]."""
    x = codes[table.long()].float() * scales[table.long()][..., None, None]
    return x.transpose(-4, -3).flatten(-3, -2)


def _shared(s):
    hq, hkv, d, n, page = s["hq"], s["hkv"], s["d"], s["q"], s["page"]
    g, y, b0 = hq // hkv, [], 0
    for prefix, of in zip(s["prefix_list"], s["of"]):
        pre = prefix // page
        q = s["queries"][b0 * n:(b0 + of) * n].float().view(of, n, hkv, g, d) * (1.0 / math.sqrt(d))
        lens = s["lens"][b0:b0 + of].long() - prefix
        mine = s["table"][b0:b0 + of, pre:pre + -(-s["max_own"] // page)]
        k, v = (_pages(c, z, mine) for c, z in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
        x = q.permute(0, 2, 3, 1, 4).flatten(2, 3) @ k.transpose(2, 3)  # [of, hkv, g n, L]
        last = lens[:, None] - n + torch.arange(n, device="cuda")  # each token's own position
        hidden = torch.arange(k.shape[2], device="cuda") > last[:, :, None]
        x = x.unflatten(2, (g, n)).masked_fill(hidden[:, None, None], -math.inf).flatten(2, 3)
        k1, v1 = (_pages(c, z, s["table"][b0, :pre]) for c, z in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
        x1 = q.permute(2, 0, 3, 1, 4).flatten(1, 3) @ k1.transpose(1, 2)  # [hkv, of g n, P]
        top1 = x1.amax(-1).view(hkv, of, g * n).transpose(0, 1)
        top = torch.maximum(x.amax(-1), top1)
        x = torch.exp(x - top[..., None])
        x1 = torch.exp(x1 - top.transpose(0, 1).flatten(1, 2)[..., None])
        total = x.sum(-1) + x1.sum(-1).view(hkv, of, g * n).transpose(0, 1)
        z = x @ v + (x1 @ v1).view(hkv, of, g * n, d).transpose(0, 1)
        z = (z / total[..., None]).view(of, hkv, g, n, d).permute(0, 3, 1, 2, 4).reshape(of * n, hq, d)
        y.append(z)
        b0 += of
    y = torch.cat(y)
    if s["gates"] is not None:
        y = y / (1.0 + torch.exp(-s["gates"].float()))
    return y.bfloat16()


# --------------------------------------------------------------------- run
def run(state):
    s = state
    if not own:
        return {"tables": _tables, "verify": _verify, "shared": _shared}[s["op"]](s)
    import nvfp4_weight_quantized_gemv_gb300 as nv
    if s["op"] == "tables":
        out = nv.nvfp4_kv_tables(s["table"], s["held"], s["pages"], s["span"], s["lens"], s["new"], s["page"], s["tokens"])
        return (*out, s["table"], s["pages"])
    if s["op"] == "verify":
        return nv.nvfp4_verify_drafts(s["target"], s["tokens"], s["cu"], s["u"], s["pick"], draft=s["draft"],
                                      kv_lens=s["lens"])
    return nv.nvfp4_attn_paged_shared(s["queries"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["lens"],
                                      s["group_cu"], s["prefixes"], s["q"], max_kv_len=s["max_kv"],
                                      max_group_tokens=s["max_group"], max_own_len=s["max_own"], gate=s["gates"])


def work(case):
    c = case
    if c["op"] == "tables":
        kv, q = _table_lengths(c)
        held = _table_held(c, kv)
        t, moved = sum(q), sum(abs(-(-(n + m) // c["page"]) - h) for n, m, h in zip(kv, q, held))
        # lengths and pages held in and out, cu_q; pages between ring and tables; a page number, position and slot a token
        return {"bytes": c["b"] * 24 + moved * 8 + t * 12 + sum(-(-m // c["page"]) for m in q) * 4, "flops": 8 * c["b"] + 4 * t}
    if c["op"] == "verify":
        n = [max(0, c["drafts"] - int(c["drafts"] * f * 0.7)) if c["ragged"] else c["drafts"] for f in _spread(c["b"])]
        rows = 2 if c["given"] else 1  # read whole: the row that the new token is drawn from, of both distributions
        return {"bytes": c["b"] * rows * c["vocab"] * 4 + sum(n) * 20 + c["b"] * 24, "flops": c["b"] * 2 * rows * c["vocab"]}
    prefix, of, mine = _shared_lengths(c)
    hq, hkv, d, q = c["hq"], c["hkv"], c["d"], c["q"]
    codes = sum(prefix) + sum(mine)
    pairs = sum(p * n * q for p, n in zip(prefix, of)) + sum(q * m - q * (q - 1) // 2 for m in mine)
    return {"bytes": 2 * codes * hkv * d + -(-codes // c["page"]) * hkv * 8 + c["b"] * q * hq * d * (6 if c["gate"] else 4),
            "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------- exact
def _exact_tables(c, s):
    """One request after the other, on the host."""
    table, held, pages = s["table"].tolist(), s["held"].tolist(), s["pages"].tolist()
    kv, new, (head, tail) = s["lens"].tolist(), s["new"].tolist(), s["span"].tolist()
    page, ring, room = c["page"], len(pages), s["tokens"]
    free = [pages[i % ring] for i in range(head, tail)]
    used, asked, asked_pages, back = 0, 0, 0, []
    cu, pos, slot, lens = [0], [], [], []
    for b in range(c["b"]):
        ok = kv[b] >= 0 and new[b] >= 0 and kv[b] + new[b] <= len(table[b]) * page
        asked += new[b] if ok else 0
        ok = ok and (new[b] == 0 or asked <= room)
        need = -(-(kv[b] + new[b]) // page)
        asked_pages += max(0, need - held[b]) if ok else 0
        ok = ok and (need <= held[b] or asked_pages <= len(free))
        if ok:
            while held[b] < need:
                table[b][held[b]] = free[used]
                used, held[b] = used + 1, held[b] + 1
            back += table[b][need:held[b]]
            held[b] = need
            for p in range(kv[b], kv[b] + new[b]):
                pos.append(p)
                slot.append(table[b][p // page] * page + p % page)
        cu.append(len(pos))
        lens.append(kv[b] + (new[b] if ok else 0))
    for i, p in enumerate(back):
        pages[(tail + i) % ring] = p
    rest = room - len(pos)
    return (_ints(cu), _ints(lens), _ints(pos + [0] * rest), _ints(slot + [-1] * rest, torch.int64), _ints(held),
            _ints([head + used, tail + len(back)], torch.int64), _ints(table), _ints(pages))


def _exact_verify(c, s):
    """One sequence after the other; a row's cumulative sums in 64 bits."""
    cu, tokens, u, pick, lens = (s[k].tolist() for k in ("cu", "tokens", "u", "pick", "lens"))
    out, count, new, left = [], [], [], []
    for b in range(c["b"]):
        row, n = cu[b], 0
        while row + 1 < cu[b + 1]:
            x = tokens[row + 1]
            q = s["draft"][row, x].item() if c["given"] else 1.0
            if not u[row] * q < s["target"][row, x].item():
                break
            out.append(x)
            row, n = row + 1, n + 1
        weights = s["target"][row].cpu().double()
        whole = weights.clone()
        if row + 1 < cu[b + 1]:
            if c["given"]:
                weights = torch.relu(weights - s["draft"][row].cpu().double())
            else:
                weights[tokens[row + 1]] = 0
        if not (weights > 0).any():
            weights = whole
        total = torch.cumsum(weights, 0)
        at = int(torch.searchsorted(total, pick[b] * total[-1:], right=True))
        at = min(at, int(weights.nonzero()[-1]))
        out += [at] + [-1] * (cu[b + 1] - row - 1)
        count.append(n)
        new.append(at)
        left.append(lens[b] - (cu[b + 1] - 1 - row))
    return _ints(out), _ints(count), _ints(new), _ints(left)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "tables":
        return _exact_tables(c, s)
    if c["op"] == "verify":
        return _exact_verify(c, s)
    g, n = c["hq"] // c["hkv"], c["q"]
    y = torch.empty(s["queries"].shape, dtype=torch.float64, device="cuda")
    for b, kv in enumerate(s["lens"].tolist()):
        pages = s["table"][b, :-(-kv // c["page"])].long()
        hidden = torch.arange(kv, device="cuda") > torch.arange(kv - n, kv, device="cuda")[:, None]
        for h in range(c["hkv"]):
            k, v = ((x[pages, h].double() * z[pages, h].double()[:, None, None]).flatten(0, 1)[:kv]
                    for x, z in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            rows = s["queries"][b * n:(b + 1) * n, h * g:(h + 1) * g].double()
            z = torch.einsum("nge,le->gnl", rows, k) / math.sqrt(c["d"])
            w = torch.softmax(z.masked_fill(hidden, -math.inf), -1)
            y[b * n:(b + 1) * n, h * g:(h + 1) * g] = torch.einsum("gnl,le->nge", w, v)
    return y if s["gates"] is None else y * torch.sigmoid(s["gates"].double())


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(8)]:
        print(case, work(case))
