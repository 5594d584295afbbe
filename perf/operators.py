"""Measured cases of the key/value cache operators: append, read, attention and attention with a shared prefix.

The cache is paged and group-quantised: one row of `head_dim` values of one token and head is held as
`nbits`-wide codes and, for each group of `group_size` values, an fp16 scale and zero point, and stands
for (code - zero) * scale.  `run` computes the operators in elementary torch operations, or calls the framework
where `own` is set.
"""
import math
import random

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
FP16_MAX = 65504.0
SCALE_MIN = 2.0 ** -24      # the smallest positive fp16
FLAT = 2.0 ** -10           # a group's step is at least this fraction of its largest magnitude


def listed():
    return [
        # the new token of one sequence, at each layer of each decoding step: latency
        {"name": "append 1 token", "op": "append", "tokens": 1, "kv_heads": 8, "head_dim": 128, "nbits": 4,
         "group": 64, "type": "bf16", "page": 64, "fused": True},
        # a mixed batch of prompt pieces and single tokens, a small head, 8-bit codes
        {"name": "append 1003 tokens", "op": "append", "tokens": 1003, "kv_heads": 8, "head_dim": 64, "nbits": 8,
         "group": 32, "type": "fp16", "page": 16, "fused": False},
        # the prompt of a decoder with 32 heads of its own (4096 wide)
        {"name": "append 8192 tokens", "op": "append", "tokens": 8192, "kv_heads": 32, "head_dim": 128, "nbits": 4,
         "group": 64, "type": "bf16", "page": 64, "fused": True},
        # a few hundred tokens read back to be moved or requantised, wide head, 2-bit codes
        {"name": "read 257 tokens", "op": "read", "tokens": 257, "kv_heads": 2, "head_dim": 256, "nbits": 2,
         "group": 128, "type": "fp16", "page": 32},
        # a long context read back
        {"name": "read 32768 tokens", "op": "read", "tokens": 32768, "kv_heads": 8, "head_dim": 128, "nbits": 4,
         "group": 64, "type": "bf16", "page": 64},
        # one short conversation: latency
        {"name": "attend 1 x 131", "op": "attend", "batch": 1, "nq": 1, "length": 131, "ragged": False,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "nbits": 4, "group": 64, "type": "bf16", "page": 64, "window": 0},
        # 16 conversations of uneven length, 32 heads of their own
        {"name": "attend 16 x 2048 ragged", "op": "attend", "batch": 16, "nq": 1, "length": 2048, "ragged": True,
         "heads": 32, "kv_heads": 32, "head_dim": 128, "nbits": 4, "group": 64, "type": "fp16", "page": 16, "window": 0},
        # a full serving batch with shared key heads
        {"name": "attend 64 x 4096", "op": "attend", "batch": 64, "nq": 1, "length": 4096, "ragged": False,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "nbits": 4, "group": 64, "type": "bf16", "page": 64, "window": 0},
        # one very long document, 8-bit codes
        {"name": "attend 1 x 131072", "op": "attend", "batch": 1, "nq": 1, "length": 131072, "ragged": False,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "nbits": 8, "group": 128, "type": "bf16", "page": 128, "window": 0},
        # five drafted tokens checked at once, behind a sliding window, odd lengths
        {"name": "attend 7 x 5 windowed", "op": "attend", "batch": 7, "nq": 5, "length": 3001, "ragged": True,
         "heads": 15, "kv_heads": 3, "head_dim": 64, "nbits": 2, "group": 32, "type": "fp16", "page": 32, "window": 1000},
        # a handful of requests behind one instruction text that ends inside a page
        {"name": "prefix 8 x 1000", "op": "prefix", "batch": 8, "nq": 1, "prefix": 1000, "length": 77, "ragged": True,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "nbits": 4, "group": 64, "type": "fp16", "page": 64},
        # a full batch of questions about one long document
        {"name": "prefix 64 x 32768", "op": "prefix", "batch": 64, "nq": 1, "prefix": 32768, "length": 400, "ragged": True,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "nbits": 4, "group": 64, "type": "bf16", "page": 64},
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    head_dim = rng.choice([64, 128, 128, 256])
    case = {"op": rng.choice(["append", "read", "attend", "attend", "prefix"]), "head_dim": head_dim,
            "nbits": rng.choice([2, 4, 4, 8]), "group": rng.choice([g for g in (32, 64, 128) if g <= head_dim]),
            "type": rng.choice(["fp16", "bf16"]), "page": rng.choice([16, 32, 64, 128]),
            "kv_heads": rng.choice([1, 2, 3, 4, 8, 16])}
    row = case["kv_heads"] * head_dim
    if case["op"] in ("append", "read"):
        case["tokens"] = _spread(rng, 1, min(40000, 2 ** 25 // row))
        if case["op"] == "append":
            case["fused"] = rng.random() < 0.5
        return case
    case["heads"] = case["kv_heads"] * rng.choice([1, 2, 3, 4, 5, 7, 8])
    case["nq"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
    case["ragged"] = rng.random() < 0.7
    if case["op"] == "attend":
        case["batch"] = _spread(rng, 1, 48)
        case["length"] = _spread(rng, 1, min(120000, 2 ** 26 // (row * case["batch"])))
        case["window"] = rng.choice([0, 0, 0, _spread(rng, 1, 5000)])
    else:
        case["nq"] = rng.choice([1, 1, 1, 2, 4])
        case["heads"] = case["kv_heads"] * rng.choice([1, 2, 4, 5])
        rows = case["heads"] * case["nq"]
        case["batch"] = _spread(rng, 2, max(2, min(64, 2048 // rows)))
        case["prefix"] = _spread(rng, 1, min(32000, 2 ** 25 // row))
        case["length"] = _spread(rng, case["nq"], max(case["nq"], min(1000, 2 ** 25 // (row * case["batch"]))))
    return case


def _lengths(case):
    """The tokens of each sequence of the batch: a property of the case, not of the seed."""
    if not case["ragged"]:
        return [case["length"]] * case["batch"]
    rng = random.Random("%d %d %d" % (case["batch"], case["length"], case["nq"]))
    return [case["length"]] + [rng.randint(min(case["nq"], case["length"]), case["length"]) for _ in range(case["batch"] - 1)]


# ---------------------------------------------------------------- inputs

def _values(gen, tokens, heads, dim, offset):
    """Projected keys or values: normal, with a few channels that are larger and off centre (as keys have)."""
    x = torch.randn(tokens, heads, dim, generator=gen, device="cuda")
    gain = torch.exp(0.5 * torch.randn(heads, dim, generator=gen, device="cuda"))
    return x * gain + offset * torch.randn(heads, dim, generator=gen, device="cuda") * gain


def _interleave(x, group, pieces):
    """[..., D] in element order -> the order in which a row is stored: pieces outermost, then groups."""
    n = x.shape[-1] // group
    return x.unflatten(-1, (n, pieces, group // pieces)).transpose(-3, -2).flatten(-3)


def _in_order(x, group, pieces):
    n = x.shape[-1] // group
    return x.unflatten(-1, (pieces, n, group // pieces)).transpose(-3, -2).flatten(-3)


def _quantize(x, nbits, group):
    """Codes [..., D] (uint8) and metadata [..., D/g, 2] (fp16 scale and zero) of rows x, in binary32."""
    top = float(2 ** nbits - 1)
    x = x.float().clamp(-FP16_MAX, FP16_MAX).unflatten(-1, (-1, group))
    lo, hi = x.amin(-1), x.amax(-1)
    least = torch.maximum(lo.abs(), hi.abs()) * FLAT
    scale = torch.maximum((hi - lo) / torch.full_like(lo, top), least).clamp_min(SCALE_MIN).half()
    inv = 1.0 / scale.float()
    zero = (-lo * inv).half()
    code = torch.round(x * inv[..., None] + zero.float()[..., None]).clamp(0.0, top)
    return code.flatten(-2).to(torch.uint8), torch.stack((scale, zero), -1)


def _pack(code, nbits):
    per = 8 // nbits
    code = code.unflatten(-1, (-1, per))
    out = code[..., 0].clone()
    for i in range(1, per):
        out |= code[..., i] << (nbits * i)
    return out


def _unpack(data, nbits):
    shift = torch.arange(0, 8, nbits, device=data.device, dtype=torch.uint8)
    return ((data[..., None] >> shift) & (2 ** nbits - 1)).flatten(-2)


def _dequantize(data, meta, nbits, group, pieces):
    """Rows in binary32 from packed codes [..., D*b/8] and metadata [..., D/g, 2]."""
    code = _in_order(_unpack(data, nbits), group, pieces).float().unflatten(-1, (-1, group))
    meta = meta.float()
    return ((code - meta[..., 1:2]) * meta[..., 0:1]).flatten(-2)


def _empty_cache(case, pages):
    h, p, d, g = case["kv_heads"], case["page"], case["head_dim"], case["group"]
    cache = {}
    for name in ("k", "v"):
        cache[name + "_codes"] = torch.zeros(pages, h, p, d * case["nbits"] // 8, dtype=torch.uint8, device="cuda")
        cache[name + "_meta"] = torch.zeros(pages, h, p, d // g, 2, dtype=torch.float16, device="cuda")
    return cache


def _filled_cache(case, gen, pages):
    """A cache whose every slot holds a quantised row."""
    cache = _empty_cache(case, pages)
    h, p, d = case["kv_heads"], case["page"], case["head_dim"]
    step = max(1, 2 ** 25 // (h * p * d))
    for name, pieces, offset in (("k", 4, 1.0), ("v", 8, 0.2)):
        for a in range(0, pages, step):
            n = min(step, pages - a)
            x = _values(gen, n * p, h, d, offset).to(TYPES[case["type"]])
            code, meta = _quantize(x, case["nbits"], case["group"])
            data = _pack(_interleave(code, case["group"], pieces), case["nbits"])
            cache[name + "_codes"][a:a + n] = data.unflatten(0, (n, p)).transpose(1, 2)
            cache[name + "_meta"][a:a + n] = meta.unflatten(0, (n, p)).transpose(1, 2)
    return cache


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = TYPES[case["type"]]
    state = {"case": dict(case)}
    if case["op"] in ("append", "read"):
        n, h, d, p = case["tokens"], case["kv_heads"], case["head_dim"], case["page"]
        pages = -(-n // p) + 3
        # tokens go to (or come from) the slots of a pool's pages, which lie anywhere
        order = torch.randperm(pages, generator=gen, device="cuda")[:-(-n // p)]
        slots = (order[:, None] * p + torch.arange(p, device="cuda")).flatten()[:n].contiguous()
        if n > 3:
            slots[n // 2] = -1      # a token of the padding
        state["slots"] = slots
        if case["op"] == "read":
            state.update(_filled_cache(case, gen, pages))
            return state
        state.update(_empty_cache(case, pages))
        k, v = _values(gen, n, h, d, 1.0).to(t), _values(gen, n, h, d, 0.2).to(t)
        if case["fused"]:           # slices of the one product that gives queries, keys and values
            both = torch.cat((torch.zeros_like(k), k, v), 1)
            k, v = both[:, h:2 * h], both[:, 2 * h:]
        state["k"], state["v"] = k, v
        return state
    lens, p = _lengths(case), case["page"]
    wide = -(-max(lens) // p)
    shared = -(-case["prefix"] // p) if case["op"] == "prefix" else 0
    total = shared + sum(-(-n // p) for n in lens) + 1
    state.update(_filled_cache(case, gen, total))
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    pages = torch.zeros(len(lens), wide, dtype=torch.int32, device="cuda")
    at = shared
    for b, n in enumerate(lens):
        used = -(-n // p)
        pages[b, :used] = order[at:at + used]
        at += used
    state["pages"], state["lens"] = pages, torch.tensor(lens, dtype=torch.int32, device="cuda")
    if shared:
        state["prefix_pages"] = order[:shared].contiguous()
    state["q"] = (1.5 * torch.randn(case["batch"], case["nq"], case["heads"], case["head_dim"], generator=gen, device="cuda")).to(t)
    return state


# ---------------------------------------------------------------- one pass

def _cache(state):
    """The handle that a user's program keeps beside its cache tensors."""
    if "handle" not in state:
        from free_weight_quantization_b200 import hqq
        c = state["case"]
        state["handle"] = hqq.KVCache(state["k_codes"], state["v_codes"], state["k_meta"], state["v_meta"], c["nbits"], c["group"])
    return state["handle"]


def _run_own(state):
    from free_weight_quantization_b200 import hqq
    case, cache = state["case"], _cache(state)
    if case["op"] == "append":
        k, v = hqq.hqq_kv_append(cache, state["k"], state["v"], state["slots"], return_values=True)
        return _appended(state, k, v)
    if case["op"] == "read":
        k, v = hqq.hqq_kv_read(cache, state["slots"], dtype=TYPES[case["type"]])
        return {"k": k, "v": v}
    if case["op"] == "attend":
        out, lse = hqq.hqq_kv_attention(cache, state["q"], state["pages"], state["lens"], window=case["window"], return_lse=True)
    else:
        out, lse = hqq.hqq_kv_prefix_attention(cache, state["q"], state["prefix_pages"], case["prefix"], state["pages"],
                                               state["lens"], return_lse=True)
    return {"out": out, "lse": lse}


def _appended(state, k, v):
    return {"k": k, "v": v, "k_codes": state["k_codes"], "v_codes": state["v_codes"], "k_meta": state["k_meta"],
            "v_meta": state["v_meta"]}


def _append(state):
    case = state["case"]
    page, at = state["slots"] // case["page"], state["slots"] % case["page"]
    kept = state["slots"] >= 0
    out = []
    for name, pieces in (("k", 4), ("v", 8)):
        code, meta = _quantize(state[name], case["nbits"], case["group"])
        data = _pack(_interleave(code, case["group"], pieces), case["nbits"])
        state[name + "_codes"][page[kept], :, at[kept]] = data[kept]
        state[name + "_meta"][page[kept], :, at[kept]] = meta[kept]
        x = _dequantize(data, meta, case["nbits"], case["group"], pieces)
        out.append(torch.where(kept[:, None, None], x, 0.0).to(TYPES[case["type"]]))
    return _appended(state, *out)


def _read(state):
    case, out = state["case"], []
    slots = state["slots"].clamp_min(0)
    page, at = slots // case["page"], slots % case["page"]
    for name, pieces in (("k", 4), ("v", 8)):
        x = _dequantize(state[name + "_codes"][page, :, at], state[name + "_meta"][page, :, at], case["nbits"], case["group"], pieces)
        out.append(torch.where((state["slots"] >= 0)[:, None, None], x, 0.0).to(TYPES[case["type"]]))
    return {"k": out[0], "v": out[1]}


def _context(state, pages):
    """Keys and values in binary32 of the pages [..., n] of a table: [..., heads, n * page, D]."""
    case, out = state["case"], []
    for name, pieces in (("k", 4), ("v", 8)):
        x = _dequantize(state[name + "_codes"][pages], state[name + "_meta"][pages], case["nbits"], case["group"], pieces)
        out.append(x.transpose(-4, -3).flatten(-3, -2))
    return out


def _softmax(s):
    """exp(s - lse) and lse over the last axis; a row with nothing visible has weights of zero and lse = -inf."""
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m.isinf(), 0.0, m))
    l = e.sum(-1, keepdim=True)
    return e / torch.where(l == 0.0, 1.0, l), (torch.log(l) + m).squeeze(-1)


def _attend(state):
    case = state["case"]
    b, n, d, kv = case["batch"], case["nq"], case["head_dim"], case["kv_heads"]
    share = case["heads"] // kv
    # [B, kv, nq * share, D]: the rows that read one key head
    q = state["q"].float().unflatten(2, (kv, share)).permute(0, 2, 1, 3, 4).flatten(2, 3) * d ** -0.5
    k, v = _context(state, state["pages"].long())
    t = torch.arange(k.shape[2], device="cuda")
    lens = state["lens"].long()[:, None]
    at = lens - n + torch.arange(n, device="cuda")            # [B, nq]: each query's position among its own tokens
    seen = t <= at[..., None]
    if case.get("window"):
        seen &= t > at[..., None] - case["window"]
    s = q @ k.transpose(-1, -2)
    s = torch.where(seen.repeat_interleave(share, 1)[:, None], s, -math.inf)
    if case["op"] == "prefix":
        pk, pv = _context(state, state["prefix_pages"].long())
        pk, pv = pk[:, :case["prefix"]], pv[:, :case["prefix"]]
        rows = q.transpose(0, 1).flatten(1, 2)                 # [kv, B * nq * share, D]
        ps = (rows @ pk.transpose(-1, -2)).unflatten(1, (b, -1)).transpose(0, 1)
        w, lse = _softmax(torch.cat((ps, s), -1))
        pw = w[..., :case["prefix"]].transpose(0, 1).flatten(1, 2)
        o = (pw @ pv).unflatten(1, (b, -1)).transpose(0, 1) + w[..., case["prefix"]:] @ v
    else:
        w, lse = _softmax(s)
        o = w @ v
    o = o.unflatten(2, (n, share)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = lse.unflatten(2, (n, share)).permute(0, 2, 1, 3).flatten(2, 3)
    return {"out": o.to(TYPES[case["type"]]), "lse": lse.contiguous()}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return _append(state) if op == "append" else _read(state) if op == "read" else _attend(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    h, d = case["kv_heads"], case["head_dim"]
    held = 2 * h * (d * case["nbits"] // 8 + 4 * (d // case["group"]))     # a token's codes and metadata
    if case["op"] in ("append", "read"):
        n, values = case["tokens"], 2 * 2 * h * d                          # a token's keys and values, 16 bits each
        if case["op"] == "append":
            return {"bytes": n * (2 * values + held + 8), "flops": n * 2 * h * d * 8}
        return {"bytes": n * (values + held + 8), "flops": n * 2 * h * d * 2}
    b, n = case["batch"], case["nq"]
    lens, rows = _lengths(case), 0
    read = 0
    for m in lens:
        first = max(0, m - n + 1 - case["window"]) if case.get("window") else 0
        read += m - first
        for i in range(n):
            at = m - n + 1 + i
            rows += max(0, min(at, case["window"]) if case.get("window") else at)
    small = b * n * case["heads"] * (2 * 2 * d + 4) + 4 * (b + sum(-(-m // case["page"]) for m in lens))
    if case["op"] == "prefix":
        read += case["prefix"]
        rows += case["prefix"] * b * n
        small += 4 * -(-case["prefix"] // case["page"])
    return {"bytes": read * held + small, "flops": 4 * d * rows * case["heads"]}


# ---------------------------------------------------------------- the operators' definitions in 64 bits

def _fl32(x):
    """One rounding to binary32 of the definition, kept in 64 bits."""
    return x.to(torch.float32).to(torch.float64)


def _exact_rows(state, name, page, offsets):
    """Element by element from the stored bytes of one page: [heads, len(offsets), D] in 64 bits."""
    case = state["case"]
    d, g, nb = case["head_dim"], case["group"], case["nbits"]
    parts = 4 if name == "k" else 8
    e = torch.arange(d, device="cuda")
    place = (e % g) // (g // parts) * (d // parts) + e // g * (g // parts) + e % (g // parts)
    byte = state[name + "_codes"][page][:, offsets][..., place * nb // 8].to(torch.int64)
    code = (byte >> (place * nb % 8)) % (1 << nb)
    meta = state[name + "_meta"][page][:, offsets].to(torch.float64)[:, :, e // g]
    return (code.to(torch.float64) - meta[..., 1]) * meta[..., 0]


def _exact_append(state):
    case = state["case"]
    nb, g, d, p = case["nbits"], case["group"], case["head_dim"], case["page"]
    top, outs = (1 << nb) - 1, {}
    e = torch.arange(d, device="cuda")
    kept = torch.nonzero(state["slots"] >= 0).squeeze(1)
    for name, parts in (("k", 4), ("v", 8)):
        x = state[name].to(torch.float64).clamp(-FP16_MAX, FP16_MAX)
        n, h, _ = x.shape
        x = x.reshape(n, h, d // g, g)
        lo, hi = x.min(-1).values, x.max(-1).values
        step = _fl32(_fl32(hi - lo) / top)
        floor = _fl32(torch.maximum(-lo, hi) / 1024)
        scale = torch.maximum(torch.maximum(step, floor), torch.full_like(step, 2.0 ** -24)).to(torch.float16).to(torch.float64)
        inv = _fl32(1 / scale)
        zero = _fl32(-lo * inv).to(torch.float16).to(torch.float64)
        code = torch.round(_fl32(_fl32(x * inv[..., None]) + zero[..., None])).clamp(0, top)
        hat = _fl32(_fl32(code - zero[..., None]) * scale[..., None]).reshape(n, h, d)
        hat[state["slots"] < 0] = 0
        outs[name] = hat
        place = (e % g) // (g // parts) * (d // parts) + e // g * (g // parts) + e % (g // parts)
        data = torch.zeros(n, h, d * nb // 8, dtype=torch.int64, device="cuda")
        data.index_add_(2, place * nb // 8, code.reshape(n, h, d).to(torch.int64) << (place * nb % 8))
        where = state["slots"][kept]
        codes, meta = state[name + "_codes"].clone(), state[name + "_meta"].to(torch.float64)
        codes[where // p, :, where % p] = data[kept].to(torch.uint8)
        meta[where // p, :, where % p] = torch.stack((scale, zero), -1)[kept]
        outs[name + "_codes"], outs[name + "_meta"] = codes, meta
    return {k: outs[k] for k in ("k", "v", "k_codes", "v_codes", "k_meta", "v_meta")}


def exact(case, seed):
    state = prepare(case, seed)
    p, d = case["page"], case["head_dim"]
    if case["op"] == "append":
        return _exact_append(state)
    if case["op"] == "read":
        slots, outs = state["slots"].tolist(), {}
        for name in ("k", "v"):
            x = torch.zeros(case["tokens"], case["kv_heads"], d, dtype=torch.float64, device="cuda")
            for i in range(0, len(slots), p):      # the tokens of one page
                part = torch.tensor(slots[i:i + p], device="cuda")
                some = next(s for s in slots[i:i + p] if s >= 0) // p
                rows = _exact_rows(state, name, some, part.clamp_min(some * p) - some * p).transpose(0, 1)
                x[i:i + p] = torch.where((part >= 0)[:, None, None], rows, 0.0)
            outs[name] = _fl32(x)
        return outs
    lens, n, kv = _lengths(case), case["nq"], case["kv_heads"]
    share, every = case["heads"] // kv, torch.arange(p, device="cuda")
    shared = case.get("prefix", 0)

    def rows_of(name, table, count):
        return torch.cat([_exact_rows(state, name, i, every) for i in table], 1)[:, :count] if table else \
            torch.zeros(kv, 0, d, dtype=torch.float64, device="cuda")

    head = {name: rows_of(name, state["prefix_pages"].tolist() if shared else [], shared) for name in ("k", "v")}
    out = torch.zeros(case["batch"], n, case["heads"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], n, case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, m in enumerate(lens):
        table = state["pages"][b, :-(-m // p)].tolist()
        k, v = (torch.cat((head[name], rows_of(name, table, m)), 1) for name in ("k", "v"))
        for i in range(n):
            end = shared + m - n + i + 1
            first = max(0, end - case["window"]) if case.get("window") else 0
            if end <= first:
                continue
            q = state["q"][b, i].to(torch.float64).view(kv, share, d) / math.sqrt(d)
            s = torch.einsum("hgd,htd->hgt", q, k[:, first:end])
            z = torch.logsumexp(s, -1)
            lse[b, i] = z.flatten()
            out[b, i] = torch.einsum("hgt,htd->hgd", torch.exp(s - z[..., None]), v[:, first:end]).reshape(-1, d)
    return {"out": out, "lse": lse}
