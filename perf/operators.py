"""Measured cases of the operators around the 4-bit linear layer: the layer
with its epilogue, the expert router, and the products grouped by expert.

Four kinds of case, by their ``op``:

* ``linear``: ``linear_fused`` - one packed layer with bias, activation
  (plain, or gated: the first half of the rows is the gate, the second the
  values it multiplies) and residual, one rounding to fp16;
* ``route``: ``route_experts`` - the ``k`` largest of ``E`` logits per token,
  their softmax weights, and the tokens' slots sorted by expert;
* ``experts``: ``linear_experts`` - every routed row through its own expert's
  packed layer (ragged sizes, rows gathered from the tokens), same epilogue;
* ``combine``: ``combine_experts`` - the routed rows through their experts'
  second layer, weighted and added up per token, plus a residual.

Without ``own`` the operators run in a plain form of elementary torch
operations in 32 bits; with it they are the calls of this package.
"""
import math

import torch

own = False

DEVICE = "cuda"
ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the attention output projection of a 7B block for one token, added to the residual stream: latency
        _linear("o_proj 1 token", 1, 4096, 4096, residual=True),
        # gate and up of a 7B block in one launch for one token, the MLP's activation in the epilogue
        _linear("gate_up 1 token", 1, 22016, 4096, act="silu", gated=True),
        # the down projection of a 7B block for an odd decode batch, with a bias, added to the residual stream
        _linear("down 13 tokens", 13, 4096, 11008, bias=True, residual=True),
        # a symmetric layer with a bias and a plain activation for a ragged batch
        _linear("up gelu 61 tokens", 61, 11008, 4096, g=64, zp=False, act="gelu_tanh", bias=True),
        # prefill of the 70B-shaped MLP's first half: gate and up in one product
        _linear("gate_up 70b prefill", 2048, 57344, 8192, act="silu", gated=True),
        # one decode step's router
        _route("route 1 token", 1, 8, 2, "float16"),
        # the router of a long prompt over many experts
        _route("route 16384 tokens", 16384, 128, 8, "float32"),
        # one token through its two of eight experts: two 7B-sized gate_up layers
        _experts("gate_up 1 token 2 of 8", 1, 8, 2, 22016, 4096, act="silu", gated=True),
        # a decode batch over many small experts: a few rows for each
        _experts("gate_up 48 tokens 6 of 64", 48, 64, 6, 2816, 2048, g=64, act="silu", gated=True),
        # a ragged prompt over eight experts: a few hundred rows for each
        _experts("gate_up 1000 tokens 2 of 8", 1000, 8, 2, 22016, 4096, act="silu", gated=True),
        # the second half of the one-token and of the prompt's expert layers
        _combine("down 1 token 2 of 8", 1, 8, 2, 4096, 11008, residual=True),
        _combine("down 1000 tokens 2 of 8", 1000, 8, 2, 4096, 11008, residual=True),
    ]


def _linear(name, M, N, K, g=128, zp=True, act="none", gated=False, bias=False, residual=False):
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "g": g, "zp": zp, "act": act, "gated": gated,
            "bias": bias, "residual": residual}


def _route(name, T, E, k, dtype, renormalize=True):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "dtype": dtype, "renormalize": renormalize}


def _experts(name, T, E, k, N, K, g=128, zp=True, act="none", gated=False, bias=False):
    return {"name": name, "op": "experts", "T": T, "E": E, "k": k, "N": N, "K": K, "g": g, "zp": zp, "act": act,
            "gated": gated, "bias": bias}


def _combine(name, T, E, k, N, K, g=128, zp=True, bias=False, residual=False):
    return {"name": name, "op": "combine", "T": T, "E": E, "k": k, "N": N, "K": K, "g": g, "zp": zp, "bias": bias,
            "residual": residual}


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _size(rng, unit, lo, hi):
    """An odd multiple of ``unit`` or of a few times its double, between lo and hi."""
    unit <<= rng.randint(0, 2 if unit <= 128 else 1)
    times = 2 * _spread(rng, max(1, lo // (2 * unit)), max(1, hi // (2 * unit))) - 1
    return unit * times


def draw(rng):
    op = rng.choice(("linear", "linear", "route", "experts", "combine"))
    if op == "route":
        E = rng.choice((8, 16, 60, 64, 128, 200, 256))
        c = _route("", _spread(rng, 1, 16384), E, rng.randint(1, min(8, E)), rng.choice(("float16", "float32")),
                   rng.random() < 0.7)
    else:
        g = rng.choice((32, 64, 128, 128, 128, 256))
        zp = rng.random() < 0.7
        act = rng.choice(ACTIVATIONS)
        gated = rng.random() < 0.5
        unit = 16 if gated and op != "combine" else 8
        if op == "linear":
            M, K = _spread(rng, 1, 2048), _size(rng, g, 512, 11008)
            N = _size(rng, unit, 512, 28672)
            c = _linear("", M, N, K, g, zp, act, gated, rng.random() < 0.5, rng.random() < 0.5)
        else:
            T, E = _spread(rng, 1, 1000), rng.choice((8, 8, 16, 60, 64))
            k = rng.randint(1, 2 if E == 8 else 6)
            top = 11008 if E <= 16 else 2816
            K = _size(rng, g, 512, 4096 if op == "experts" else top)
            N = _size(rng, unit, 512, top if op == "experts" else 4096)
            if op == "experts":
                c = _experts("", T, E, k, N, K, g, zp, act, gated, rng.random() < 0.3)
            else:
                c = _combine("", T, E, k, N, K, g, zp, rng.random() < 0.3, rng.random() < 0.5)
    del c["name"]
    return c


# --------------------------------------------------------------- the inputs
def _rand_words(shape, gen):
    return torch.randint(-(1 << 31), 1 << 31, shape, generator=gen, device=DEVICE, dtype=torch.int32)


def _packed(lead, N, K, g, zp, gen):
    """A packed weight as the package stores it, with codes spread like a quantized Gaussian's: each code the sum of
    two 3-bit numbers and a bit, zero points 6 to 9, and scales that give weights of variance about 1 / K."""
    words = lead + (N, K // 8)
    qweight = (_rand_words(words, gen) & 0x77777777) + (_rand_words(words, gen) & 0x77777777)
    qweight += _rand_words(words, gen) & 0x11111111
    G = K // g
    scales = torch.rand(lead + (N // 8, G, 8), generator=gen, device=DEVICE) * 0.5 + 0.75
    scales = (scales / (3.3 * math.sqrt(K))).to(torch.float16)
    qzeros = (_rand_words(lead + (N // 8, G), gen) & 0x33333333) + 0x66666666 if zp else None
    return qweight, scales, qzeros


def _activations(rows, K, gen):
    """Standard normal, with 1% of the channels 20 times as large in every row."""
    x = torch.randn((rows, K), generator=gen, device=DEVICE)
    hot = torch.randperm(K, generator=gen, device=DEVICE)[: max(1, round(0.01 * K))]
    x[:, hot] *= 20.0
    return x.to(torch.float16)


def _logits(T, E, gen):
    """Logits of a router with favoured experts: unit noise on a per-expert offset."""
    return torch.randn((T, E), generator=gen, device=DEVICE) + 0.5 * torch.randn((1, E), generator=gen, device=DEVICE)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "route":
        s["logits"] = _logits(case["T"], case["E"], gen).to(getattr(torch, case["dtype"]))
        return s
    N, K, g, zp = case["N"], case["K"], case["g"], case["zp"]
    lead = () if case["op"] == "linear" else (case["E"],)
    s["packed"] = _packed(lead, N, K, g, zp, gen) + ((N, K, g, zp) if case["op"] == "linear" else lead + (N, K, g, zp))
    s["bias"] = torch.randn(lead + (N,), generator=gen, device=DEVICE).to(torch.float16) if case["bias"] else None
    rows = case["M"] if case["op"] == "linear" else case["T"]
    if case["op"] != "linear":
        s["route"] = _plain_route(_logits(rows, case["E"], gen), case["k"], True)
    s["x"] = _activations(rows * case["k"] if case["op"] == "combine" else rows, K, gen)
    width = N // 2 if case.get("gated") else N
    s["residual"] = (torch.randn((rows, width), generator=gen, device=DEVICE).to(torch.float16)
                     if case.get("residual") else None)
    return s


# ----------------------------------------------------------------- one pass
def run(s):
    if own:
        import bit_weight_only_awq_amd as awq

        if s["op"] == "linear":
            return awq.linear_fused(s["x"], awq.PackedWeight(*s["packed"]), bias=s["bias"], activation=s["act"],
                                    gated=s["gated"], residual=s["residual"])
        if s["op"] == "route":
            return tuple(awq.route_experts(s["logits"], s["k"], s["renormalize"]))
        experts, route = awq.PackedExperts(*s["packed"]), awq.ExpertRoute(*s["route"])
        if s["op"] == "experts":
            return awq.linear_experts(s["x"], experts, route, bias=s["bias"], activation=s["act"], gated=s["gated"])
        return awq.combine_experts(s["x"], experts, route, bias=s["bias"], residual=s["residual"])
    if s["op"] == "linear":
        acc = s["x"].float() @ _plain_weight(*s["packed"]).t()
        return _plain_epilogue(acc, s["bias"], s["act"], s["gated"], s["residual"]).to(torch.float16)
    if s["op"] == "route":
        return _plain_route(s["logits"], s["k"], s["renormalize"])
    if s["op"] == "experts":
        slots = s["route"][3].long()
        acc, used = _plain_grouped(s["x"][slots // s["k"]], s["packed"], s["route"][2])
        return _plain_epilogue(acc, _of_rows(s["bias"], used), s["act"], s["gated"], None).to(torch.float16)
    acc, used = _plain_grouped(s["x"], s["packed"], s["route"][2])
    acc = _plain_epilogue(acc, _of_rows(s["bias"], used), "none", False, None)
    weights, positions = s["route"][1], s["route"][4].long()
    y = (acc[positions] * weights.unsqueeze(-1)).sum(1)
    return (y if s["residual"] is None else y + s["residual"].float()).to(torch.float16)


# ---------------------------------------------------------- the plain forms
def _plain_weight(qweight, scales, qzeros, *rest):
    """(q - z) * s in 32 bits, [..., N, K]."""
    N, K, g, zp = rest[-4:]
    lead = qweight.shape[:-2]
    at = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=qweight.device, dtype=torch.int32)
    q = (((qweight.unsqueeze(-1) >> at) & 15).float()).view(*lead, N, K // g, g)
    s = scales.float().transpose(-1, -2).reshape(*lead, N, K // g, 1)
    z = 8.0
    if zp:
        at = torch.arange(0, 32, 4, device=qweight.device, dtype=torch.int32)
        z = ((qzeros.unsqueeze(-1) >> at) & 15).float().transpose(-1, -2).reshape(*lead, N, K // g, 1)
    return ((q - z) * s).view(*lead, N, K)


def _plain_activation(v, act):
    if act == "relu":
        return torch.clamp(v, min=0.0)
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_epilogue(acc, bias, act, gated, residual):
    if bias is not None:
        acc = acc + bias.float()
    if gated:
        gate, up = acc.chunk(2, dim=-1)
        acc = _plain_activation(gate, act) * up
    else:
        acc = _plain_activation(acc, act)
    return acc if residual is None else acc + residual.float()


def _plain_route(logits, k, renormalize):
    """(ids, weights, offsets, rows, positions): per token its k largest logits (the lower index first among equal
    ones) and their softmax weights; slot t * k + j of token t sorted by expert, then by slot; each slot's place."""
    v = logits.float()
    top, ids = torch.sort(v, dim=-1, descending=True, stable=True)
    ids = ids[:, :k]
    e = torch.exp(v - top[:, :1])
    weights = e.gather(1, ids)
    weights = weights / (weights if renormalize else e).sum(-1, keepdim=True)
    flat = ids.reshape(-1)
    rows = torch.sort(flat, stable=True)[1]
    places = torch.empty_like(rows)
    places[rows] = torch.arange(rows.numel(), device=rows.device)
    counts = (flat.unsqueeze(0) == torch.arange(v.shape[1], device=v.device).unsqueeze(1)).sum(1)
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    i32 = torch.int32
    return ids.to(i32), weights, offsets.to(i32), rows.to(i32), places.view(ids.shape).to(i32)


def _plain_grouped(x, packed, offsets):
    """Row r of x through the weight of the expert whose range of offsets holds r; and each row's expert. The rows of
    the experts that have any are padded to one length and multiplied in one batched product."""
    E = packed[-5]
    counts = offsets[1:] - offsets[:-1]
    used = counts.nonzero().flatten()
    experts = torch.repeat_interleave(torch.arange(E, device=x.device), counts.long())
    nth = torch.repeat_interleave(torch.arange(used.numel(), device=x.device), counts[used].long())
    within = torch.arange(x.shape[0], device=x.device) - offsets[experts].long()
    padded = x.new_zeros((used.numel(), int(counts.max()), x.shape[1]), dtype=torch.float32)
    padded[nth, within] = x.float()
    qweight, scales, qzeros = packed[:3]
    w = _plain_weight(qweight[used], scales[used], None if qzeros is None else qzeros[used], *packed[3:])
    return torch.matmul(padded, w.transpose(-1, -2))[nth, within], experts


def _of_rows(bias, experts):
    return None if bias is None else bias[experts]


# ------------------------------------------------------ what a pass must do
def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        slots = T * k
        return {"bytes": T * E * (2 if case["dtype"] == "float16" else 4) + 16 * slots + 4 * (E + 1),
                "flops": 3 * T * E}
    N, K, g = case["N"], case["K"], case["g"]
    weight = N * K / 2 + N * (K // g) * (2.5 if case["zp"] else 2) + (2 * N if case["bias"] else 0)
    width = N // 2 if case.get("gated") else N
    if case["op"] == "linear":
        M = case["M"]
        return {"bytes": weight + 2 * M * K + 2 * M * width * (2 if case["residual"] else 1), "flops": 2 * M * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    used = E * (1.0 - (1.0 - k / E) ** T)  # of E experts, under even routing
    slots = T * k
    if case["op"] == "experts":
        data = 2 * T * K + 2 * slots * width + 4 * slots
    else:
        data = 2 * slots * K + 2 * T * N * (2 if case["residual"] else 1) + 8 * slots
    return {"bytes": used * weight + data, "flops": 2 * slots * N * K}


# ---------------------------------------------------- the same, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s["logits"].double(), case["k"], case["renormalize"])
    if case["op"] == "linear":
        y = _exact_rows(s["x"].double(), s["packed"], None, s["bias"], s["act"], s["gated"])
        return y if s["residual"] is None else y + s["residual"].double()
    offsets, slots, k = s["route"][2].tolist(), s["route"][3].long(), case["k"]
    gather = case["op"] == "experts"
    parts = []
    for e in range(case["E"]):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            x = s["x"][torch.div(slots[lo:hi], k, rounding_mode="floor") if gather else slice(lo, hi)].double()
            parts.append(_exact_rows(x, s["packed"], e, s["bias"], case.get("act", "none"), case.get("gated", False)))
    rows = torch.cat(parts)
    if gather:
        return rows
    y = torch.zeros((case["T"], case["N"]), dtype=torch.float64, device=DEVICE)
    weighted = rows * s["route"][1].double().reshape(-1)[slots].unsqueeze(1)
    y.index_add_(0, torch.div(slots, k, rounding_mode="floor"), weighted)
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_rows(x, packed, expert, bias, act, gated):
    """x (64 bits) through one packed weight and its epilogue, a block of output channels at a time."""
    qweight, scales, qzeros = (t if t is None or expert is None else t[expert] for t in packed[:3])
    N, K, g, _ = packed[-4:]
    k = torch.arange(K, device=DEVICE)
    c = k % 8
    place, group = 16 * (c % 2) + 4 * torch.div(c, 2, rounding_mode="floor"), torch.div(k, g, rounding_mode="floor")
    out = torch.empty((x.shape[0], N), dtype=torch.float64, device=DEVICE)
    for lo in range(0, N, 8192):
        n = torch.arange(lo, min(N, lo + 8192), device=DEVICE)
        words = qweight[n].long().repeat_interleave(8, dim=1)
        code = torch.bitwise_right_shift(words, place).bitwise_and(15).double()
        octet, row = torch.div(n, 8, rounding_mode="floor"), n % 8
        scale = scales[octet, :, row].double()[:, group]
        if qzeros is None:
            zero = 8.0
        else:
            zero = torch.bitwise_right_shift(qzeros[octet].long(), (4 * row).unsqueeze(1)).bitwise_and(15)
            zero = zero.double()[:, group]
        out[:, lo : lo + n.numel()] = torch.mm(x, ((code - zero) * scale).t().contiguous())
    if bias is not None:
        out += (bias if expert is None else bias[expert]).double()
    half = N // 2
    v = out[:, :half] if gated else out
    if act == "relu":
        v = torch.where(v > 0, v, torch.zeros_like(v))
    elif act == "silu":
        v = v * torch.special.expit(v)
    elif act == "gelu":
        v = v * torch.special.ndtr(v)
    elif act == "gelu_tanh":
        v = v * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v**3))
    return v * out[:, half:] if gated else v


def _exact_route(v, k, renormalize):
    """Only the weights are computed numbers: the rest is whole."""
    T, E = v.shape
    left, picked = v.clone(), []
    index = torch.arange(E, device=DEVICE)
    for _ in range(k):
        best = left.max(dim=1, keepdim=True).values
        at = torch.where(left == best, index, E).min(dim=1, keepdim=True).values
        picked.append(at)
        left.scatter_(1, at, -math.inf)
    ids = torch.cat(picked, dim=1)
    chosen = v.gather(1, ids)
    among = chosen if renormalize else v
    return None, torch.exp(chosen - torch.logsumexp(among, dim=1, keepdim=True)), None, None, None
