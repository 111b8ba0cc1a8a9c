"""The operators of a 4-bit decode step, as cases to be timed and compared.

Four operators: products of a few tokens with MXFP4 / NVFP4 weights, writing
keys and values into a paged MXFP4 cache, attention over that cache, and
copying its pages.  Each has a plain form in elementary torch operations (32
bits, rounded once at the end), the framework's own call, and a definition in
64 bits.

Formats.  MXFP4: 32 consecutive values share a power of two 2^(byte - 127),
elements are E2M1 nibbles, element 2j in the low nibble of byte j.  NVFP4: 16
values share an E4M3 scale, times one fp32 scale of the tensor.  A cache page
is one run of bytes with four sections: K codes [heads, page, dim / 2], V codes
[heads, page / 16, dim / 2, 16], then K's and V's scales, each [heads, page / 16,
dim / 32, 16]; where the last axis is 16 it counts tokens.
"""
import math

import torch

own = False
DEVICE = "cuda"

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # One token through the smallest projection: a call's own cost.
        {"name": "mx matvec 1x256x512", "op": "matvec", "kind": "mx", "tokens": 1, "n": 256, "k": 512, "out": "bf16"},
        # One token through a square projection, the ordinary decode step.
        {"name": "mx matvec 1x8192x8192", "op": "matvec", "kind": "mx", "tokens": 1, "n": 8192, "k": 8192, "out": "bf16"},
        # A few tokens checked at once, odd rows, logits kept in fp32.
        {"name": "nv matvec 5x4097x7168", "op": "matvec", "kind": "nv", "tokens": 5, "n": 4097, "k": 7168, "out": "f32"},
        # A full decode batch through a fused gate and up projection.
        {"name": "mx matvec 64x16384x7168", "op": "matvec", "kind": "mx", "tokens": 64, "n": 16384, "k": 7168, "out": "bf16"},
        # One short chat: the smallest attention call.
        {"name": "attention 1 seq decode", "op": "attention", "seqs": 1, "tokens": 1, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "shortest": 1000, "longest": 1000, "window": 0, "causal": True, "lse": False},
        # A full decode batch over long ragged contexts: bound by the cache's bytes.
        {"name": "attention 64 seqs decode", "op": "attention", "seqs": 64, "tokens": 1, "q_heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "shortest": 4096, "longest": 8192, "window": 0, "causal": True, "lse": False},
        # Drafted tokens verified under a sliding window, small pages, every query head
        # with its own keys; slots of the batch that are empty or shorter than the draft.
        {"name": "attention 7 seqs verify", "op": "attention", "seqs": 7, "tokens": 4, "q_heads": 8, "kv_heads": 8, "dim": 64,
         "page": 16, "shortest": 0, "longest": 5001, "window": 1024, "causal": True, "lse": True},
        # A chunk of a long prompt over what the cache already holds: bound by arithmetic.
        {"name": "attention 2 seqs chunk", "op": "attention", "seqs": 2, "tokens": 512, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "shortest": 12000, "longest": 16384, "window": 0, "causal": True, "lse": True},
        # The new token of every sequence of a batch; the values stored come back too.
        {"name": "append 33 decode", "op": "append", "tokens": 33, "kv_heads": 8, "q_heads": 32, "dim": 128, "page": 64,
         "pages": 600, "run": 1, "values": True},
        # A prompt's keys and values, consecutive slots.
        {"name": "append 16384 prompt", "op": "append", "tokens": 16384, "kv_heads": 8, "q_heads": 32, "dim": 128, "page": 64,
         "pages": 600, "run": 16384, "values": False},
        # The last pages of eight forked sequences, four layers.
        {"name": "copy 8 pages", "op": "copy", "layers": 4, "pages": 64, "copies": 8, "kv_heads": 8, "dim": 128, "page": 16},
        # Compacting a cache: many pages of all layers move.
        {"name": "copy 512 pages", "op": "copy", "layers": 8, "pages": 1536, "copies": 512, "kv_heads": 8, "dim": 128, "page": 64},
    ]


def spread(rng, lo, hi):
    """A whole number of lo..hi, evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("matvec", "matvec", "attention", "attention", "append", "copy"))
    if op == "matvec":
        kind = rng.choice(("mx", "nv"))
        step = 32 if kind == "mx" else 16
        return {"op": op, "kind": kind, "tokens": spread(rng, 1, 64), "n": spread(rng, 64, 16384), "k": step * spread(rng, 8, 7168 // step),
                "out": rng.choice(("bf16", "bf16", "f32"))}
    if op == "attention":
        heads, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 5, 8))
        case = {"op": op, "seqs": spread(rng, 1, 64), "tokens": rng.choice((1, 1, spread(rng, 2, 8), spread(rng, 9, 512))),
                "q_heads": heads * group, "kv_heads": heads, "dim": rng.choice((64, 96, 128, 128, 192, 256)), "page": rng.choice((16, 32, 48, 64, 128)),
                "shortest": 0, "longest": spread(rng, 16, 16384), "window": rng.choice((0, 0, spread(rng, 16, 4096))),
                "causal": rng.random() < 0.8, "lse": rng.random() < 0.5}
        while case["seqs"] > 1 and (case["seqs"] * case["longest"] * heads * case["dim"] > 1 << 28
                                    or case["seqs"] * case["longest"] * case["tokens"] * heads * group * case["dim"] > 1 << 35):
            case["seqs"] //= 2
        case["shortest"] = rng.choice((0, case["longest"] // 2, case["longest"]))
        return case
    if op == "append":
        n, page, dim = spread(rng, 1, 16384), rng.choice((16, 32, 48, 64, 128)), rng.choice((64, 96, 128, 128, 192, 256))
        heads = rng.choice((1, 2, 4, 8))
        n = min(n, (1 << 24) // (heads * dim))
        run = max(rng.choice((1, n, spread(rng, 1, n))), n // 1024)
        # every run starts on a page of its own
        return {"op": op, "tokens": n, "kv_heads": heads, "q_heads": heads * rng.choice((1, 4)), "dim": dim, "page": page,
                "pages": -(-n // run) * (-(-run // page) + 1) + spread(rng, 1, 64), "run": run, "values": rng.random() < 0.5}
    copies = spread(rng, 1, 256)
    return {"op": op, "layers": spread(rng, 1, 8), "pages": 2 * copies + spread(rng, 1, 256), "copies": copies, "kv_heads": rng.choice((1, 2, 4, 8)),
            "dim": rng.choice((64, 96, 128, 192, 256)), "page": rng.choice((16, 32, 48, 64))}


# -- formats ------------------------------------------------------------------


def page_sections(heads, dim, page):
    """Where the four sections of a page begin, and the page's bytes."""
    codes, scales = heads * page * dim // 2, heads * page * dim // 32
    return 0, codes, 2 * codes, 2 * codes + scales, 2 * (codes + scales)


def e2m1_code(x):
    """E2M1 code (0..15) of fp32 values already divided by their scale: nearest, ties to even, saturating."""
    a = x.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8) + (a >= 1.75).to(torch.uint8)
            + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8))
    return code + 8 * torch.signbit(x).to(torch.uint8)


def e2m1_value(codes):
    """fp32 values of E2M1 codes."""
    mag = (codes & 7).float()
    big = torch.where(mag < 4, 0.5 * mag, torch.where(mag < 6, mag - 2, 2 * mag - 8))
    return torch.where(codes >= 8, -big, big)


def power(byte):
    """fp32 2^(byte - 127), NaN for 255."""
    v = torch.exp2(byte.double() - 127).float()
    return torch.where(byte == 255, torch.full_like(v, math.nan), v)


def mx_quantize(x):
    """fp32 [..., d] -> E2M1 codes [..., d], E8M0 bytes [..., d / 32]."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    amax = g.abs().amax(-1)
    byte = (torch.frexp(amax)[1] - 1 - 2 + 127).clamp(0, 254)
    byte = torch.where(amax == 0, torch.zeros_like(byte), byte).to(torch.uint8)
    code = e2m1_code(g * torch.exp2(127 - byte.double()).float()[..., None])
    return code.reshape(x.shape), byte


def nv_quantize(x):
    """fp32 [n, k] -> E2M1 codes [n, k], E4M3 bytes [n, k / 16], fp32 [1]."""
    g = x.reshape(x.shape[0], -1, 16)
    scale = x.abs().amax() / 2688
    s = (g.abs().amax(-1) / (6 * scale)).clamp(max=448).to(torch.float8_e4m3fn)
    eff = (s.float() * scale)[..., None]
    code = e2m1_code(torch.where(eff > 0, g / torch.where(eff > 0, eff, torch.ones_like(eff)), torch.zeros_like(g)))
    return code.reshape(x.shape), s.view(torch.uint8), scale.reshape(1)


def pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def unpack(byte):
    return torch.stack((byte & 15, byte >> 4), -1).flatten(-2)


# -- inputs -------------------------------------------------------------------


def generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(seed)


def normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEVICE)


def prepare(case, seed):
    g = generator(seed)
    state = dict(case)
    if case["op"] == "matvec":
        # weights as they come from a checkpoint, a few outliers among them; normalised activations
        w = 0.02 * normal(g, case["n"], case["k"])
        w = torch.where(torch.rand(w.shape, generator=g, device=DEVICE) < 1e-3, 20 * w, w).bfloat16().float()
        state["x"] = normal(g, case["tokens"], case["k"]).bfloat16()
        code, state["s"], *rest = (mx_quantize if case["kind"] == "mx" else nv_quantize)(w)
        state["q"], state["g"] = pack(code), rest[0] if rest else None
        state["out_dtype"] = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        return state
    heads, dim, page = case["kv_heads"], case["dim"], case["page"]
    at = page_sections(heads, dim, page)
    if case["op"] == "copy":
        state["cache"] = torch.randint(0, 256, (case["layers"], case["pages"], at[4]), generator=g, device=DEVICE, dtype=torch.uint8)
        order = torch.randperm(case["pages"], generator=g, device=DEVICE).int()
        state["src"], state["dst"] = order[:case["copies"]].clone(), order[case["copies"]:2 * case["copies"]].clone()
        return state
    if case["op"] == "append":
        # keys and values as views of a fused projection's output
        qkv = normal(g, case["tokens"], (case["q_heads"] + 2 * heads) * dim).bfloat16()
        k, v = qkv[:, case["q_heads"] * dim:].view(case["tokens"], 2 * heads, dim).split(heads, 1)
        run, n = case["run"], case["tokens"]
        each = -(-run // page) + 1  # pages of a run, which may begin inside its first
        order = torch.randperm(case["pages"], generator=g, device=DEVICE)
        begin = torch.randint(0, page, (-(-n // run),), generator=g, device=DEVICE)
        i = torch.arange(n, device=DEVICE)
        pos = begin[i // run] + i % run
        slots = order[(i // run) * each + pos // page] * page + pos % page
        state.update(k=k, v=v, slots=slots, cache=torch.zeros(case["pages"], at[4], device=DEVICE, dtype=torch.uint8))
        return state
    seqs, longest = case["seqs"], case["longest"]
    width = -(-longest // page)
    pages = seqs * width
    lengths = torch.randint(case["shortest"], longest + 1, (seqs,), generator=g, device=DEVICE).int()
    if case["shortest"] == 0 and seqs > 2:
        lengths[0], lengths[1] = 0, min(2, longest)
    cache = torch.empty(pages, at[4], device=DEVICE, dtype=torch.uint8)
    spikes = 1 + 3 * (torch.rand(heads, 1, dim, generator=g, device=DEVICE) < 0.03).float()  # a few strong channels, as keys have
    code, byte = mx_quantize((normal(g, pages, heads, page, dim) * spikes).bfloat16().float())
    blocks = (pages, heads, page // 16, 16, -1)
    cache[:, at[0]:at[1]], cache[:, at[2]:at[3]] = pack(code).flatten(1), byte.view(blocks).mT.flatten(1)
    code, byte = mx_quantize(normal(g, pages, heads, page, dim).bfloat16().float())
    cache[:, at[1]:at[2]], cache[:, at[3]:] = pack(code).view(blocks).mT.flatten(1), byte.view(blocks).mT.flatten(1)
    state["q"] = normal(g, seqs, case["tokens"], case["q_heads"], dim).bfloat16()
    state["table"] = torch.randperm(pages, generator=g, device=DEVICE).int().view(seqs, width)
    state.update(cache=cache, lengths=lengths, scale=dim ** -0.5)
    return state


# -- the operators --------------------------------------------------------------


def run(state):
    return {"matvec": matvec, "attention": attention, "append": append, "copy": copy}[state["op"]](state)


def matvec(st):
    if own:
        import block_scaled_precision_mxfp8_amd as mxq

        if st["kind"] == "mx":
            return mxq.mxfp4_matvec(st["x"], st["q"], st["s"], out_dtype=st["out_dtype"])
        return mxq.nvfp4_matvec(st["x"], st["q"], st["s"], st["g"], out_dtype=st["out_dtype"])
    s = power(st["s"]) if st["kind"] == "mx" else st["s"].view(torch.float8_e4m3fn).float() * st["g"]
    w = e2m1_value(unpack(st["q"]))
    w = (w.view(*s.shape, -1) * s[..., None]).view(w.shape)
    return (st["x"].float() @ w.t()).to(st["out_dtype"])


def plain_cache(st):
    """fp32 keys and values [seqs, heads, width * page, dim] of the state's sequences."""
    heads, dim, page = st["kv_heads"], st["dim"], st["page"]
    at = page_sections(heads, dim, page)
    rows = st["cache"][st["table"].long()]
    seqs, width = st["table"].shape
    flat = (seqs, heads, width * page)
    part = rows[..., at[0]:at[1]].view(seqs, width, heads, page, dim // 2).transpose(1, 2)
    s = power(rows[..., at[2]:at[3]].view(seqs, width, heads, page // 16, dim // 32, 16).mT.transpose(1, 2)).reshape(seqs, heads, width, page, -1)
    k = (e2m1_value(unpack(part)).unflatten(-1, (-1, 32)) * s[..., None]).reshape(*flat, dim)
    part = rows[..., at[1]:at[2]].view(seqs, width, heads, page // 16, dim // 2, 16).mT.transpose(1, 2)
    s = power(rows[..., at[3]:].view(seqs, width, heads, page // 16, dim // 32, 16).mT.transpose(1, 2))
    v = (e2m1_value(unpack(part)).unflatten(-1, (-1, 32)) * s[..., None]).reshape(*flat, dim)
    return k, v


def attention(st):
    if own:
        import block_scaled_precision_mxfp8_amd as mxq

        return mxq.mxfp4_kv_attention(st["q"], st["cache"], st["table"], st["lengths"], st["kv_heads"], st["page"], scale=st["scale"],
                                      causal=st["causal"], window=st["window"], return_lse=st["lse"])
    k, v = plain_cache(st)
    seqs, tokens, heads, dim = st["q"].shape
    group = heads // st["kv_heads"]
    q = st["q"].float().view(seqs, tokens, -1, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, -1, group * tokens, dim)
    score = (torch.matmul(q, k.mT.contiguous()) * st["scale"]).view(seqs, -1, group, tokens, k.shape[2])
    length = st["lengths"].view(-1, 1, 1)
    j = torch.arange(k.shape[2], device=DEVICE)
    at = length - tokens + torch.arange(tokens, device=DEVICE).view(-1, 1)
    seen = (j < length).expand(seqs, tokens, -1)
    if st["causal"]:
        seen = seen & (j <= at)
    if st["window"]:
        seen = seen & (j > at - st["window"])
    seen = seen[:, None, None]
    top = torch.where(seen, score, -math.inf).amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.where(seen, torch.exp(score - top), 0.0)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    out = torch.matmul(p.view(seqs, -1, group * tokens, p.shape[-1]), v).view(seqs, -1, group, tokens, dim)
    out = out.permute(0, 3, 1, 2, 4).reshape(seqs, tokens, heads, dim).bfloat16()
    if not st["lse"]:
        return out
    lse = (top + torch.log(total))[..., 0]
    return out, lse.permute(0, 3, 1, 2).reshape(seqs, tokens, heads)


def append(st):
    if own:
        import block_scaled_precision_mxfp8_amd as mxq

        values = mxq.mxfp4_kv_append(st["cache"], st["k"], st["v"], st["slots"], st["page"], fake_quant=st["values"])
        return (st["cache"], *values) if st["values"] else st["cache"]
    cache, page, slots = st["cache"], st["page"], st["slots"]
    heads, dim = st["kv_heads"], st["dim"]
    at = page_sections(heads, dim, page)
    where, inside = slots // page, slots % page
    code, byte = mx_quantize(st["k"].float())
    k_value = (e2m1_value(code).unflatten(-1, (-1, 32)) * power(byte)[..., None]).flatten(-2).bfloat16()
    cache[:, at[0]:at[1]].view(-1, heads, page, dim // 2)[where, :, inside] = pack(code)
    cache[:, at[2]:at[3]].view(-1, heads, page // 16, dim // 32, 16)[where, :, inside // 16, :, inside % 16] = byte
    code, byte = mx_quantize(st["v"].float())
    v_value = (e2m1_value(code).unflatten(-1, (-1, 32)) * power(byte)[..., None]).flatten(-2).bfloat16()
    cache[:, at[1]:at[2]].view(-1, heads, page // 16, dim // 2, 16)[where, :, inside // 16, :, inside % 16] = pack(code)
    cache[:, at[3]:].view(-1, heads, page // 16, dim // 32, 16)[where, :, inside // 16, :, inside % 16] = byte
    return (cache, k_value, v_value) if st["values"] else cache


def copy(st):
    if own:
        import block_scaled_precision_mxfp8_amd as mxq

        mxq.mxfp4_kv_copy_pages(st["cache"], st["src"], st["dst"])
        return st["cache"]
    st["cache"][:, st["dst"].long()] = st["cache"][:, st["src"].long()]
    return st["cache"]


# -- what a pass cannot do without ------------------------------------------------


def work(case):
    if case["op"] == "matvec":
        t, n, k = case["tokens"], case["n"], case["k"]
        scales = n * k // 32 if case["kind"] == "mx" else n * k // 16 + 4
        return {"bytes": n * k // 2 + scales + 2 * t * k + (2 if case["out"] == "bf16" else 4) * t * n, "flops": 2 * t * n * k}
    heads, dim = case["kv_heads"], case["dim"]
    token = 2 * heads * (dim // 2 + dim // 32)  # a token's keys and values in the cache
    if case["op"] == "append":
        return {"bytes": case["tokens"] * (8 + 4 * heads * dim + token + (4 * heads * dim if case["values"] else 0)), "flops": 0}
    if case["op"] == "copy":
        return {"bytes": 2 * case["layers"] * case["copies"] * case["page"] * token + 8 * case["copies"], "flops": 0}
    # lengths are uniform between shortest and longest; pairs of a query and a visible token, on average
    seqs, t, mean = case["seqs"], case["tokens"], (case["shortest"] + case["longest"]) / 2
    pairs = max(1.0, mean * t - (t * (t - 1) / 2 if case["causal"] else 0))
    reach = mean
    if case["window"]:
        pairs, reach = min(pairs, t * case["window"]), min(mean, case["window"] + t)
    rows = seqs * t * case["q_heads"]
    return {"bytes": int(seqs * reach * token + 4 * rows * dim + (4 * rows if case["lse"] else 0)),
            "flops": int(4 * seqs * case["q_heads"] * dim * pairs)}


# -- the definitions in 64 bits -----------------------------------------------------


def exact(case, seed):
    if case["op"] == "copy" or (case["op"] == "append" and not case["values"]):
        return None  # bytes alone
    st = prepare(case, seed)
    levels = torch.tensor([s * v for s in (1.0, -1.0) for v in LEVELS], dtype=torch.float64, device=DEVICE)
    if case["op"] == "matvec":
        w = torch.empty(case["n"], case["k"], dtype=torch.float64, device=DEVICE)
        w[:, 0::2], w[:, 1::2] = levels[(st["q"] % 16).long()], levels[(st["q"] // 16).long()]
        if case["kind"] == "mx":
            w *= (2.0 ** (st["s"].double() - 127)).repeat_interleave(32, 1)
        else:
            w *= (st["s"].view(torch.float8_e4m3fn).double() * st["g"].double()).repeat_interleave(16, 1)
        return torch.mm(st["x"].double(), w.t().contiguous())
    if case["op"] == "append":
        values = []
        for x in (st["k"], st["v"]):
            x = x.double().unflatten(-1, (-1, 32))
            largest = x.abs().amax(-1, keepdim=True)
            unit = torch.where(largest > 0, 2.0 ** (torch.floor(torch.log2(largest)) - 2).clamp(min=-127), torch.ones_like(largest))
            far = (x.abs()[..., None] / unit[..., None] - levels[:8]).abs()
            # the nearest level; of two as near, the one with an even code
            near = (far == far.amin(-1, keepdim=True)).double() * torch.tensor([2.0, 1.0] * 4, dtype=torch.float64, device=DEVICE)
            values.append((levels[near.argmax(-1)] * unit * torch.where(torch.signbit(x), -1.0, 1.0)).flatten(-2))
        return None, values[0], values[1]
    heads, dim, page, t, group = case["kv_heads"], case["dim"], case["page"], case["tokens"], case["q_heads"] // case["kv_heads"]
    out = torch.zeros(case["seqs"], t, case["q_heads"], dim, dtype=torch.float64, device=DEVICE)
    lse = torch.full((case["seqs"], t, case["q_heads"]), -math.inf, dtype=torch.float64, device=DEVICE)
    code_bytes, scale_bytes = heads * page * dim // 2, heads * page * dim // 32
    for b, n in enumerate(st["lengths"].tolist()):
        if n == 0:
            continue
        held = st["cache"][st["table"][b, : -(-n // page)].long()]
        kc, vc, ks, vs = held.split([code_bytes, code_bytes, scale_bytes, scale_bytes], 1)
        kc, ks = kc.reshape(-1, heads, page, dim // 2), ks.reshape(-1, heads, page // 16, dim // 32, 16).transpose(3, 4).reshape(-1, heads, page, dim // 32)
        vc = vc.reshape(-1, heads, page // 16, dim // 2, 16).transpose(3, 4).reshape(-1, heads, page, dim // 2)
        vs = vs.reshape(-1, heads, page // 16, dim // 32, 16).transpose(3, 4).reshape(-1, heads, page, dim // 32)
        pair = []
        for c, s in ((kc, ks), (vc, vs)):
            x = torch.empty(*c.shape[:3], dim, dtype=torch.float64, device=DEVICE)
            x[..., 0::2], x[..., 1::2] = levels[(c % 16).long()], levels[(c // 16).long()]
            x *= (2.0 ** (s.double() - 127)).repeat_interleave(32, 3)
            pair.append(x.transpose(0, 1).reshape(heads, -1, dim)[:, :n])
        where = n - t + torch.arange(t, device=DEVICE)[:, None]
        j = torch.arange(n, device=DEVICE)[None]
        hidden = torch.zeros(t, n, dtype=torch.bool, device=DEVICE)
        if case["causal"]:
            hidden |= j > where
        if case["window"]:
            hidden |= j <= where - case["window"]
        some = ~hidden.all(1)
        for h in range(case["q_heads"]):
            s = torch.mm(st["q"][b, :, h].double() * st["scale"], pair[0][h // group].t().contiguous())
            s = s.masked_fill(hidden, -math.inf)[some]
            lse[b, some, h] = torch.logsumexp(s, -1)
            out[b, some, h] = torch.mm(torch.softmax(s, -1), pair[1][h // group])
    return (out, lse) if case["lse"] else out
