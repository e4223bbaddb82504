"""Measured cases of the operators on a paged cache of keys and values, between
a block's 4-bit q/k/v layer and its output layer.

Three kinds of case, by their ``op``:

* ``append``: ``append_kv`` - new tokens' rows of the fused q/k/v layer: queries
  and keys rotated by their positions (one axis, or several for images), keys
  and values written to their sequences' pages, and, with ``bounds``, each
  page's lowest and highest key per channel kept up to date;
* ``attend``: ``attend`` - causal attention of the new tokens over their
  sequences' pages, ragged, with the first ``shared`` tokens of all sequences
  (a long common prompt) read and multiplied once for the whole batch;
* ``sparse``: ``select_pages`` and ``attend_pages`` - for each token and key
  head the pages whose bounds allow the largest products with the query, and
  attention over those pages only.

Without ``own`` the operators run in a plain form of elementary torch
operations in 32 bits (angles and the pages' scores in 64); with it they are
the calls of this package.
"""
import math

import torch

own = False

DEVICE = "cuda"


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a 7B block (32 heads of 128, as many key heads): latency
        _append("append 1 token", 1, (1, 1), (1000, 1000), 32, 32, 128, 16),
        # a ragged decode batch of a 70B-shaped block, eight query heads per key head, with the pages' bounds
        _append("append 61 tokens", 61, (1, 1), (0, 5000), 64, 8, 128, 32, bounds=True),
        # three prompts with images: positions along three axes, a part of the channels for each
        _append("append 3 image prompts", 3, (900, 1800), (0, 77), 64, 8, 128, 32, axes=3, bounds=True),
        # one token of a 7B block over one long conversation: no other sequence to fill the chip with
        _attend("attend 1 token of 8191", 1, (1, 1), (8190, 8190), 32, 32, 128, 16),
        # a decode batch of a 70B-shaped block, lengths from a few tokens to four thousand
        _attend("attend 48 tokens", 48, (1, 1), (7, 4000), 64, 8, 128, 32),
        # the same after a system prompt that all sequences share
        _attend("attend 61 tokens, 8192 shared", 61, (1, 1), (1, 500), 64, 8, 128, 16, shared=8192),
        # questions about one long document: a few dozen new tokens each
        _attend("attend 13 questions, 16384 shared", 13, (20, 101), (0, 30), 64, 8, 128, 32, shared=16384),
        # a 7B block's prompt, nothing before it
        _attend("attend a prompt of 2000", 1, (2000, 2000), (0, 0), 32, 32, 128, 16),
        # one token over a very long context, 128 of its 6251 pages
        _sparse("sparse 1 token of 100001", 1, (1, 1), (100000, 100000), 64, 8, 128, 16, count=128),
        # a decode batch over long contexts, 64 of up to 1024 pages each
        _sparse("sparse 32 tokens", 32, (1, 1), (9000, 32767), 64, 8, 128, 32, count=64),
    ]


def _batch(name, op, B, new, past, Hq, Hkv, D, S):
    """B sequences with new[0] to new[1] new tokens after past[0] to past[1] of their own; Hq query heads, Hkv key
    heads of D channels; pages of S tokens."""
    return {"name": name, "op": op, "B": B, "new_lo": new[0], "new_hi": new[1], "past_lo": past[0], "past_hi": past[1],
            "Hq": Hq, "Hkv": Hkv, "D": D, "S": S}


def _append(name, B, new, past, Hq, Hkv, D, S, rotary=None, axes=1, interleaved=False, bounds=False):
    return {**_batch(name, "append", B, new, past, Hq, Hkv, D, S), "rotary": D if rotary is None else rotary, "axes": axes,
            "interleaved": interleaved, "bounds": bounds}


def _attend(name, B, new, past, Hq, Hkv, D, S, shared=0):
    return {**_batch(name, "attend", B, new, past, Hq, Hkv, D, S), "shared": shared}


def _sparse(name, B, new, past, Hq, Hkv, D, S, count, first=1, recent=2):
    return {**_batch(name, "sparse", B, new, past, Hq, Hkv, D, S), "count": count, "first": first, "recent": recent}


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "attend", "sparse"))
    D = rng.choice((64, 96, 128, 128, 128, 256))
    Hkv, G = rng.choice(((30, 1), (8, 8), (8, 7), (10, 4), (5, 3), (1, 16), (1, 8), (7, 3)))
    if D == 256:
        Hkv = min(Hkv, 16)
    Hq, S = Hkv * G, rng.choice((16, 16, 32, 64, 128))
    B = _spread(rng, 1, 64)
    if op == "append":
        new = _spread(rng, 1, max(1, 4000 // B))
        past = _spread(rng, 1, 20000) - 1
        c = _append("", B, (rng.randint(1, new), new), (past // 3, past), Hq, Hkv, D, S,
                    rng.choice((D, D, D // 2, 0)), rng.choice((1, 1, 3)), rng.random() < 0.3, rng.random() < 0.5)
    elif op == "sparse":
        past = _spread(rng, 500, min(100000, 2000000 // B))
        new = rng.choice((1, 1, 1, 4))
        c = _sparse("", B, (1, new), (rng.randint(0, past), past), Hq, Hkv, D, S, max(4, _spread(rng, 64, 2048) // S))
    else:
        kind = rng.choice(("decode", "shared", "chunk"))
        if kind == "decode":
            past = _spread(rng, 1, min(30000, 150000 // B))
            c = _attend("", B, (1, rng.choice((1, 1, 1, 5))), (rng.randint(0, past), past), Hq, Hkv, D, S)
        elif kind == "shared":
            past, new = _spread(rng, 1, 600), _spread(rng, 1, max(1, 400 // B))
            shared = S * (_spread(rng, 256, 12000) // S)
            c = _attend("", B, (rng.randint(1, new), new), (past // 2, past), Hq, Hkv, D, S, shared)
        else:
            B = min(B, 6)
            new = _spread(rng, 16, 1500 // B)
            past = _spread(rng, 1, 8000) - 1
            c = _attend("", B, (rng.randint(1, new), new), (past // 2, past), Hq, Hkv, D, S)
    del c["name"]
    return c


def _ragged(n, lo, hi):
    """n whole numbers from lo to hi in no order, the first of them hi."""
    return [hi - (hi - lo) * ((i * 607) % 1009) // 1008 for i in range(n)]


def _lengths(case):
    """New tokens and length (with them) of each sequence."""
    new, past = _ragged(case["B"], case["new_lo"], case["new_hi"]), _ragged(case["B"], case["past_lo"], case["past_hi"])
    return new, [case.get("shared", 0) + p + n for p, n in zip(past, new)]


# --------------------------------------------------------------- the inputs
def _sequences(case, gen):
    """Offsets, lengths and page tables: pages in no order, those of the shared tokens the same in every table."""
    new, lengths = _lengths(case)
    S, common = case["S"], case.get("shared", 0) // case["S"]
    own_pages = [-(-n // S) - common for n in lengths]
    pool = common + sum(own_pages) + 3
    order = torch.randperm(pool, generator=gen, device=DEVICE).to(torch.int32)
    tables = torch.full((case["B"], common + max(own_pages) + 1), -1, dtype=torch.int32, device=DEVICE)
    tables[:, :common] = order[:common]
    at = common
    for b, n in enumerate(own_pages):
        tables[b, common : common + n] = order[at : at + n]
        at += n
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    i32 = {"dtype": torch.int32, "device": DEVICE}
    return (torch.tensor(offsets, **i32), torch.tensor(lengths, **i32), tables), new, lengths, pool


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    s = dict(case)
    Hq, Hkv, D, S = case["Hq"], case["Hkv"], case["D"], case["S"]
    s["seqs"], s["new"], s["lengths"], pool = _sequences(case, gen)
    T = sum(s["new"])
    half = {"generator": gen, "dtype": torch.float16, "device": DEVICE}
    s["k"] = torch.randn((pool, Hkv, S, D), **half)
    s["v"] = torch.randn((pool, Hkv, S, D), **half)
    if case["op"] == "append":
        s["qkv"] = torch.randn((T, (Hq + 2 * Hkv) * D), **half)
        R, A = case["rotary"], case["axes"]
        s["inv_freq"] = s["positions"] = s["axis"] = None
        if R:
            s["inv_freq"] = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEVICE) / R)).float()
            if A > 1:
                s["positions"] = torch.randint(0, 5000, (T, A), generator=gen, device=DEVICE, dtype=torch.int32)
                s["axis"] = (torch.arange(R // 2, device=DEVICE) * 8 // (R // 2) * 3 // 8).to(torch.int32)
        s["bounds"] = None
        if case["bounds"]:
            s["bounds"] = torch.stack((s["k"].amin(2), s["k"].amax(2)), 2)
            for b in range(case["B"]):  # pages that are filled in part
                past = s["lengths"][b] - s["new"][b]
                if past % S:
                    page = int(s["seqs"][2][b, past // S])
                    kept = s["k"][page, :, : past % S]
                    s["bounds"][page] = torch.stack((kept.amin(1), kept.amax(1)), 1)
        return s
    s["q"] = (1.5 * torch.randn((T, Hq * D), generator=gen, device=DEVICE)).to(torch.float16)
    if case["op"] == "sparse":
        s["k"] += 0.7 * torch.randn((pool, Hkv, 1, D), **half)  # neighbouring keys are alike
        s["bounds"] = torch.stack((s["k"].amin(2), s["k"].amax(2)), 2)
    return s


# ----------------------------------------------------------------- one pass
def run(s):
    if own:
        import bit_weight_only_awq_amd as awq

        cache, seqs = awq.KvCache(s["k"], s["v"], s.get("bounds")), awq.Sequences(*s["seqs"])
        if s["op"] == "append":
            q = awq.append_kv(s["qkv"], cache, seqs, s["inv_freq"], positions=s["positions"], axes=s["axis"],
                              interleaved=s["interleaved"])
            return (q, s["k"], s["v"]) + (() if s["bounds"] is None else (s["bounds"],))
        if s["op"] == "attend":
            return awq.attend(s["q"], cache, seqs, shared=s["shared"])
        pages = awq.select_pages(s["q"], cache, seqs, s["count"], first=s["first"], recent=s["recent"])
        return pages, awq.attend_pages(s["q"], cache, seqs, pages)
    if s["op"] == "append":
        return _plain_append(s)
    if s["op"] == "attend":
        return _plain_attend(s)
    return _plain_sparse(s)


# ---------------------------------------------------------- the plain forms
def _plain_tokens(s):
    """Each new token's place in its sequence, page and slot."""
    offsets, lengths, tables = s["seqs"]
    new = offsets[1:] - offsets[:-1]
    seq = torch.repeat_interleave(torch.arange(new.numel(), device=DEVICE), new.long())
    place = torch.arange(seq.numel(), device=DEVICE) - offsets[seq] + lengths[seq] - new[seq]
    return place, tables[seq, place // s["S"]].long(), place % s["S"]


def _plain_rotate(x, cos, sin, interleaved):
    R = 2 * cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., : R // 2], x[..., R // 2 : R]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., R:]), -1)


def _plain_append(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    place, page, slot = _plain_tokens(s)
    x = s["qkv"].float().view(-1, Hq + 2 * Hkv, D)
    q, k, v = x[:, :Hq], x[:, Hq : Hq + Hkv], x[:, Hq + Hkv :]
    if s["inv_freq"] is not None:
        at = place.unsqueeze(1) if s["positions"] is None else s["positions"][:, s["axis"].long()]
        angle = at.double() * s["inv_freq"].double()
        cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
        q, k = _plain_rotate(q, cos, sin, s["interleaved"]), _plain_rotate(k, cos, sin, s["interleaved"])
    q, k = q.to(torch.float16), k.to(torch.float16)
    s["k"][page, :, slot] = k
    s["v"][page, :, slot] = v.to(torch.float16)
    q = q.reshape(-1, Hq * D)
    if s["bounds"] is None:
        return q, s["k"], s["v"]
    bounds = s["bounds"].float()
    bounds[page[slot == 0]] = torch.tensor([math.inf, -math.inf], device=DEVICE).view(1, 1, 2, 1)
    index, k = page.view(-1, 1, 1).expand(k.shape), k.float()
    s["bounds"].copy_(torch.stack((bounds[:, :, 0].scatter_reduce(0, index, k, "amin"),
                                   bounds[:, :, 1].scatter_reduce(0, index, k, "amax")), 2).to(torch.float16))
    return q, s["k"], s["v"], s["bounds"]


def _plain_softmax(scores):
    e = torch.exp(scores - scores.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_attend(s):
    Hkv, D, S = s["Hkv"], s["D"], s["S"]
    G, out, t = s["Hq"] // Hkv, [], 0
    for b, (n, length) in enumerate(zip(s["new"], s["lengths"])):
        table = s["seqs"][2][b, : -(-length // S)].long()
        k = s["k"][table].transpose(0, 1).reshape(Hkv, -1, D)[:, :length].float()
        v = s["v"][table].transpose(0, 1).reshape(Hkv, -1, D)[:, :length].float()
        q = s["q"][t : t + n].float().view(n, Hkv, G, D).transpose(0, 1).reshape(Hkv, n * G, D)
        scores = torch.matmul(q, k.transpose(1, 2).contiguous()) * D**-0.5
        if n > 1:
            place = torch.arange(length - n, length, device=DEVICE).repeat_interleave(G)
            scores = torch.where(torch.arange(length, device=DEVICE) > place.unsqueeze(1), -math.inf, scores)
        y = torch.matmul(_plain_softmax(scores), v)
        out.append(y.view(Hkv, n, G, D).transpose(0, 1).reshape(n, Hkv * G * D).to(torch.float16))
        t += n
    return torch.cat(out)


def _plain_sparse(s):
    Hkv, D, S, count, first, recent = s["Hkv"], s["D"], s["S"], s["count"], s["first"], s["recent"]
    G, t = s["Hq"] // Hkv, 0
    T, head = s["q"].shape[0], torch.arange(Hkv, device=DEVICE).unsqueeze(1)
    pages = torch.full((T, Hkv, count), -1, dtype=torch.int32, device=DEVICE)
    out = []
    for b, (n, length) in enumerate(zip(s["new"], s["lengths"])):
        table = s["seqs"][2][b].long()
        for place in range(length - n, length):
            have = place // S + 1
            if have <= count:
                chosen = torch.arange(have, device=DEVICE).expand(Hkv, have)
            else:
                middle = s["bounds"][table[first : have - recent]].double()  # [pages, Hkv, 2, D]
                q = s["q"][t].double().view(Hkv, G, D)
                up, down = q.clamp(min=0).sum(1), q.clamp(max=0).sum(1)
                score = (middle[:, :, 1] * up + middle[:, :, 0] * down).sum(-1).t()
                best = torch.sort(score, dim=1, descending=True, stable=True)[1][:, : count - first - recent] + first
                chosen = torch.cat((torch.arange(first, device=DEVICE).expand(Hkv, first), torch.sort(best, dim=1)[0],
                                    torch.arange(have - recent, have, device=DEVICE).expand(Hkv, recent)), 1)
            pages[t, :, : chosen.shape[1]] = chosen.to(torch.int32)
            k = s["k"][table[chosen], head].float().view(Hkv, -1, D)
            v = s["v"][table[chosen], head].float().view(Hkv, -1, D)
            at = (chosen.unsqueeze(-1) * S + torch.arange(S, device=DEVICE)).view(Hkv, 1, -1)
            q = s["q"][t].float().view(Hkv, G, D)
            scores = torch.matmul(q, k.transpose(1, 2).contiguous()) * D**-0.5
            y = torch.matmul(_plain_softmax(torch.where(at > place, -math.inf, scores)), v)
            out.append(y.view(1, Hkv * G * D).to(torch.float16))
            t += 1
    return pages, torch.cat(out)


# ------------------------------------------------------ what a pass must do
def work(case):
    Hq, Hkv, D, S = case["Hq"], case["Hkv"], case["D"], case["S"]
    new, lengths = _lengths(case)
    T = sum(new)
    if case["op"] == "append":
        touched = sum(-(-length // S) - (length - n) // S for n, length in zip(new, lengths))
        return {"bytes": 2 * T * (2 * Hq + 4 * Hkv) * D + (4 * touched * Hkv * D if case["bounds"] else 0),
                "flops": 3 * T * (Hq + Hkv) * case["rotary"]}
    row = 4 * T * Hq * D  # queries in, results out
    if case["op"] == "attend":
        keys = case["shared"] + sum(length - case["shared"] for length in lengths)
        pairs = sum(n * (2 * length - n + 1) // 2 for n, length in zip(new, lengths))
        return {"bytes": row + 4 * keys * Hkv * D, "flops": 4 * pairs * Hq * D}
    scored, read, pairs = 0, 0, 0
    for n, length in zip(new, lengths):
        have = -(-length // S)
        if have > case["count"]:
            scored += have - case["first"] - case["recent"]
        for place in range(length - n, length):
            pairs += min(place + 1, case["count"] * S)
        read += min(length, case["count"] * S)  # at least, for tokens that choose alike
    return {"bytes": row + 4 * scored * Hkv * D + 4 * read * Hkv * D + 4 * T * Hkv * case["count"],
            "flops": 4 * pairs * Hq * D + 4 * scored * Hkv * D}


# ---------------------------------------------------- the same, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "attend":
        return torch.cat([_exact_rows(s, b, None) for b in range(case["B"])])
    s["chosen"] = _exact_choice(s)
    return None, torch.cat([_exact_rows(s, b, s["chosen"]) for b in range(case["B"])])


def _exact_append(s):
    """Rotation as a complex product, a sequence at a time."""
    Hq, Hkv, D, S, R = s["Hq"], s["Hkv"], s["D"], s["S"], s["rotary"]
    k, v = s["k"].double(), s["v"].double()
    bounds = None if s["bounds"] is None else s["bounds"].double()
    qs, t = [], 0
    for b, (n, length) in enumerate(zip(s["new"], s["lengths"])):
        x = s["qkv"][t : t + n].double().view(n, Hq + 2 * Hkv, D).clone()
        place = torch.arange(length - n, length, device=DEVICE)
        if R:
            at = place.view(n, 1).expand(n, R // 2) if s["positions"] is None else torch.gather(
                s["positions"][t : t + n].long(), 1, s["axis"].long().expand(n, R // 2))
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEVICE), at * s["inv_freq"].double()).unsqueeze(1)
            part = x[:, : Hq + Hkv, :R].reshape(n, Hq + Hkv, *((R // 2, 2) if s["interleaved"] else (2, R // 2)))
            if not s["interleaved"]:
                part = part.transpose(-1, -2)
            part = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
            if not s["interleaved"]:
                part = part.transpose(-1, -2)
            x[:, : Hq + Hkv, :R] = part.reshape(n, Hq + Hkv, R)
        qs.append(x[:, :Hq].reshape(n, Hq * D))
        for i in range((length - n) // S, -(-length // S)):
            page = int(s["seqs"][2][b, i])
            lo, hi = max(i * S, length - n), min((i + 1) * S, length)
            rows = slice(lo - (length - n), hi - (length - n))
            keys = x[rows, Hq : Hq + Hkv].transpose(0, 1)
            k[page, :, lo - i * S : hi - i * S] = keys
            v[page, :, lo - i * S : hi - i * S] = x[rows, Hq + Hkv :].transpose(0, 1)
            if bounds is not None:
                low, high = keys.min(1).values, keys.max(1).values
                if lo > i * S:
                    low, high = torch.minimum(low, bounds[page, :, 0]), torch.maximum(high, bounds[page, :, 1])
                bounds[page, :, 0], bounds[page, :, 1] = low, high
        t += n
    return (torch.cat(qs), k, v) + (() if bounds is None else (bounds,))


def _exact_choice(s):
    """The chosen pages of each token as a truth value per key head and page."""
    S, count, first, recent = s["S"], s["count"], s["first"], s["recent"]
    Hkv, D = s["Hkv"], s["D"]
    chosen, t = [], 0
    for b, (n, length) in enumerate(zip(s["new"], s["lengths"])):
        for place in range(length - n, length):
            have = place // S + 1
            if have <= count:
                chosen.append(torch.ones((Hkv, have), dtype=torch.bool, device=DEVICE))
            else:
                q = s["q"][t].double().view(Hkv, 1, -1, D)
                score = torch.empty((Hkv, have), dtype=torch.float64, device=DEVICE)
                for lo in range(0, have, 512):
                    both = s["bounds"][s["seqs"][2][b, lo : min(have, lo + 512)].long()].double().transpose(0, 1)
                    score[:, lo : lo + 512] = torch.maximum(q * both[:, :, :1], q * both[:, :, 1:]).sum((2, 3))
                score[:, :first] = math.inf
                score[:, have - recent :] = math.inf
                order = torch.argsort(score, dim=1, descending=True, stable=True)
                mask = torch.zeros((Hkv, have), dtype=torch.bool, device=DEVICE)
                chosen.append(mask.scatter_(1, order[:, :count], True))
            t += 1
    return chosen


def _exact_rows(s, b, chosen):
    """One sequence's new tokens, a key head and a few tokens at a time; with `chosen`, only those pages' keys."""
    Hkv, D, S = s["Hkv"], s["D"], s["S"]
    G, n, length = s["Hq"] // Hkv, s["new"][b], s["lengths"][b]
    t0 = sum(s["new"][:b])
    table = s["seqs"][2][b, : -(-length // S)].long()
    out = torch.empty((n, Hkv, G, D), dtype=torch.float64, device=DEVICE)
    keys = torch.arange(length, device=DEVICE)
    for h in range(Hkv):
        k, v = (s[c][table, h].double().view(-1, D)[:length] for c in ("k", "v"))
        step = max(1, (1 << 26) // (G * length))
        for i in range(0, n, step):
            j = min(n, i + step)
            q = s["q"][t0 + i : t0 + j].double().view(j - i, Hkv, G, D)[:, h].reshape(-1, D)
            scores = torch.mm(q, k.t().contiguous()).view(j - i, G, length) / math.sqrt(D)
            place = torch.arange(length - n + i, length - n + j, device=DEVICE)
            seen = keys.unsqueeze(0) <= place.unsqueeze(1)
            if chosen is not None:
                for r in range(i, j):
                    mask = chosen[t0 + r][h]
                    seen[r - i] &= torch.nn.functional.pad(mask, (0, len(table) - mask.numel()))[keys // S]
            scores = scores.masked_fill(~seen.unsqueeze(1), -math.inf)
            w = torch.exp(scores - torch.logsumexp(scores, dim=-1, keepdim=True))
            out[i:j, h] = torch.mm(w.view(-1, length), v).view(j - i, G, D)
    return out.view(n, -1)
