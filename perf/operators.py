"""Work of the decoder-layer operators around the expert stage: RMS norm with
the residual's addition, 8-bit quantisation in groups of 128, rotation of q/k
with the append to a paged cache, single-token attention over that cache, and
the 8-bit block-scaled matrix product.

Each case is a dict of plain values. ``run`` computes the operator in its
plain form (elementary torch operations in 32 bits, rounded once), or, where
``own`` is true, through the framework's public calls on the same inputs.
"""
import math

import torch

own = False

BLOCK = 128              # columns per activation scale, rows x columns per weight scale
E4M3_MAX = 448.0
MIN_AMAX = 1e-12         # a group's largest magnitude is taken as at least this
EPS = 1e-6
DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------- the cases

def norm(name, rows, hidden, dtype, residual, outputs, pad=0):
    return {"name": name, "op": "norm", "rows": rows, "hidden": hidden, "dtype": dtype, "residual": residual,
            "outputs": outputs, "pad": pad}


def quantize(name, rows, hidden, dtype, pad=0):
    return {"name": name, "op": "quantize", "rows": rows, "hidden": hidden, "dtype": dtype, "pad": pad}


def append(name, tokens, q_heads, kv_heads, dim, rotary, interleaved, dtype, cache, page, heads_first, unused=0):
    return {"name": name, "op": "append", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
            "rotary": rotary, "interleaved": interleaved, "dtype": dtype, "cache": cache, "page": page,
            "heads_first": heads_first, "unused": unused}


def attention(name, batch, max_len, ragged, q_heads, kv_heads, dim, dtype, cache, page, heads_first, empty=0):
    return {"name": name, "op": "attention", "batch": batch, "max_len": max_len, "ragged": ragged, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "cache": cache, "page": page,
            "heads_first": heads_first, "empty": empty}


def gemm(name, m, n, k, dtype):
    return {"name": name, "op": "gemm", "m": m, "n": n, "k": k, "dtype": dtype}


def listed():
    return [
        # the norm before the QKV product of one decoded token, straight to the product's 8-bit operand
        norm("norm_decode1_fp8", 1, 2560, "f16", True, "q"),
        # the norm of a prompt's tokens, 16-bit output for the router and the experts
        norm("norm_prompt8192", 8192, 5120, "bf16", True, "y"),
        # the attention output of a decode batch, quantised for the output product
        quantize("quantize_decode48", 48, 4096, "f16"),
        # the same for a prompt, rows cut from a wider buffer
        quantize("quantize_prompt6000", 6000, 8192, "bf16", 256),
        # one decode step of a padded batch: q/k/v cut from the QKV product, two unused rows
        append("append_decode16", 16, 20, 4, 128, 128, False, "f16", "f16", 16, False, 2),
        # a long prompt into an 8-bit cache, heads before tokens in a page
        append("append_prompt8191", 8191, 32, 8, 128, 128, False, "bf16", "e4m3", 64, True),
        # one user, short context: latency
        attention("attn_b1_len513", 1, 513, False, 20, 4, 128, "f16", "f16", 16, False),
        # a serving batch of mixed lengths with padding rows, 8-bit cache
        attention("attn_b64_ragged_e4m3", 64, 16000, True, 64, 8, 128, "bf16", "e4m3", 64, True, 3),
        # one user, long context: the split over the length alone fills the card
        attention("attn_b1_len131071", 1, 131071, False, 32, 4, 128, "bf16", "bf16", 32, False),
        # the QKV product of one decoded token: the weights' bytes
        gemm("gemm_m1_qkv", 1, 3584, 2560, "f16"),
        # a decode batch, ragged sizes
        gemm("gemm_m96_ragged", 96, 5000, 4240, "bf16"),
        # a prompt's output product
        gemm("gemm_m8192", 8192, 5120, 8192, "bf16"),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "append", "attention", "gemm"])
    dtype = rng.choice(["f16", "bf16"])
    if op in ("norm", "quantize"):
        hidden = log_int(rng, 64, 16384)
        if rng.random() < 0.75:
            hidden = -(-hidden // 128) * 128
        rows = log_int(rng, 1, max(1, min(16384, 8192 * 5120 // hidden)))
        pad = rng.choice([0, 0, 8, 128, 5])
        if op == "norm":
            case = norm("", rows, hidden, dtype, rng.random() < 0.7, rng.choice(["y", "q", "yq"]), pad)
        else:
            case = quantize("", rows, hidden, dtype, pad)
    elif op == "append":
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 5, 7, 8, 16])
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        tokens = log_int(rng, 1, max(1, min(16384, 8191 * 48 * 128 // ((heads + 2 * kv) * dim))))
        case = append("", tokens, heads, kv, dim, rng.choice([dim, dim, dim // 2]), rng.random() < 0.3, dtype,
                      rng.choice([dtype, "e4m3"]), rng.choice([1, 16, 24, 64, 256]), rng.random() < 0.5,
                      rng.choice([0, 0, tokens // 8]))
    elif op == "attention":
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 5, 7, 8, 16, 24])
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        cache = rng.choice([dtype, "e4m3"])
        batch = log_int(rng, 1, 256)
        most = 4 * 131071 * 4 * 128 * 2 // (batch * kv * dim * (1 if cache == "e4m3" else 2))
        case = attention("", batch, log_int(rng, 1, max(1, min(131072, most))), rng.random() < 0.6, heads, kv, dim,
                         dtype, cache, rng.choice([1, 16, 24, 64, 256]), rng.random() < 0.5,
                         rng.choice([0, 0, batch // 8]))
    else:
        n, k = log_int(rng, 128, 16384), 16 * log_int(rng, 8, 1024)
        if rng.random() < 0.6:
            n, k = -(-n // 128) * 128, -(-k // 128) * 128
        m = log_int(rng, 1, max(1, min(8192, 8192 * 5120 * 8192 // (n * k))))
        case = gemm("", m, n, k, dtype)
    del case["name"]
    return case


def lengths(case):
    """The sequences' lengths: all the longest, or spread over the range, the last `empty` rows of the batch unused."""
    n = case["batch"]
    lens = [case["max_len"]] * n
    if case["ragged"]:
        lens = [max(1, int(case["max_len"] * ((i * 0.6180339887498949 + 1.0) % 1.0 or 1.0))) for i in range(n)]
        lens[0] = case["max_len"]
    for i in range(case["empty"]):
        lens[n - 1 - i] = 0
    return lens


def work(case):
    op = case["op"]
    size = {"f16": 2, "bf16": 2, "e4m3": 1}
    if op in ("norm", "quantize"):
        n, w = case["rows"] * case["hidden"], size[case["dtype"]]
        scales = case["rows"] * -(-case["hidden"] // BLOCK) * 4
        if op == "quantize":
            return {"bytes": n * (w + 1) + scales, "flops": 3 * n}
        b = n * w + case["hidden"] * w + (2 * n * w if case["residual"] else 0)
        b += n * w if "y" in case["outputs"] else 0
        b += n + scales if "q" in case["outputs"] else 0
        return {"bytes": b, "flops": 6 * n}
    if op == "append":
        w, c, t, d = size[case["dtype"]], size[case["cache"]], case["tokens"], case["dim"]
        kept = t - case["unused"]
        b = t * case["q_heads"] * d * 2 * w + kept * case["kv_heads"] * d * 2 * (w + c) + t * (case["rotary"] * 4 + 12)
        return {"bytes": b, "flops": 3 * (t * case["q_heads"] + kept * case["kv_heads"]) * case["rotary"]}
    if op == "attention":
        total, d = sum(lengths(case)), case["dim"]
        b = 2 * total * case["kv_heads"] * d * size[case["cache"]]
        b += 2 * case["batch"] * case["q_heads"] * d * size[case["dtype"]] + case["batch"] * case["q_heads"] * 4
        return {"bytes": b, "flops": 4 * total * case["q_heads"] * d}
    m, n, k = case["m"], case["n"], case["k"]
    kb = -(-k // BLOCK)
    return {"bytes": m * k + n * k + 4 * kb * (m + -(-n // BLOCK)) + m * n * size[case["dtype"]], "flops": 2 * m * n * k}


# ------------------------------------------------------------------ the inputs

def normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std


def rows_of(g, case):
    """Hidden states with a few channels much larger than the others, rows cut from a buffer `pad` columns wider."""
    n, h = case["rows"], case["hidden"]
    gain = torch.exp(normal(g, h, std=0.5))
    wide = torch.zeros((n, h + case["pad"]), device=DEV, dtype=TYPES[case["dtype"]])
    wide[:, :h] = normal(g, n, h) * gain
    return wide[:, :h]


def pages_of(case, n_tokens):
    return max(1, -(-n_tokens // case["page"]))


def cache_of(case, n_pages, g=None, std=1.0):
    """A cache [pages][page][kv heads][dim], as a view of the order that it has in memory."""
    page, heads, d, t = case["page"], case["kv_heads"], case["dim"], TYPES[case["cache"]]
    shape = (n_pages, heads, page, d) if case["heads_first"] else (n_pages, page, heads, d)
    if g is None:
        c = torch.zeros(shape, device=DEV, dtype=torch.float32).to(t)
    else:
        c = torch.empty(shape, device=DEV, dtype=t)
        step = max(1, (1 << 26) // (page * heads * d))
        for i in range(0, n_pages, step):
            c[i:i + step] = normal(g, *c[i:i + step].shape, std=std).to(t)
    return c.transpose(1, 2) if case["heads_first"] else c


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    dt = TYPES[case["dtype"]]
    op = case["op"]
    if op in ("norm", "quantize"):
        n, h = case["rows"], case["hidden"]
        s["x"] = rows_of(g, case)
        if op == "norm":
            s["weight"] = (1.0 + normal(g, h, std=0.2)).to(dt)
            if case["residual"]:
                s["residual_in"] = normal(g, n, h, std=2.0).to(dt)
                s["residual"] = torch.empty_like(s["residual_in"])
        if op == "norm" and "y" in case["outputs"]:
            s["y"] = torch.empty((n, h), device=DEV, dtype=dt)
        if op == "quantize" or "q" in case["outputs"]:
            s["q"] = torch.empty((n, h), device=DEV, dtype=torch.float8_e4m3fn)
            s["scales"] = torch.empty((n, -(-h // BLOCK)), device=DEV, dtype=torch.float32)
    elif op == "append":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        qkv = normal(g, t, hq + 2 * hk, d).to(dt)
        s["q_in"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["q"] = torch.empty((t, hq, d), device=DEV, dtype=dt)
        top = t + 1000
        s["positions"] = (torch.arange(t, device=DEV) + torch.randint(0, 1000, (1,), generator=g, device=DEV)).to(torch.int32)
        freq = 10000.0 ** (-torch.arange(0, case["rotary"], 2, device=DEV, dtype=torch.float64) / case["rotary"])
        angle = torch.arange(top, device=DEV, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        pages = pages_of(case, t) + 3
        s["k_cache"], s["v_cache"] = cache_of(case, pages), cache_of(case, pages)
        order = torch.randperm(pages, generator=g, device=DEV)
        at = torch.arange(t, device=DEV)
        s["slots"] = order[at // case["page"]] * case["page"] + at % case["page"]
        if case["unused"]:
            s["slots"][t - case["unused"]:] = -1
        s["k_scale"], s["v_scale"] = (0.02, 0.015) if case["cache"] == "e4m3" else (1.0, 1.0)
        s["status"] = torch.zeros(1, device=DEV, dtype=torch.int32)
    elif op == "attention":
        b, hq, hk, d = case["batch"], case["q_heads"], case["kv_heads"], case["dim"]
        lens = lengths(case)
        need = [pages_of(case, n) for n in lens]
        total = sum(need) + 1
        quant = case["cache"] == "e4m3"
        s["k_cache"] = cache_of(case, total, g, std=50.0 if quant else 1.0)
        s["v_cache"] = cache_of(case, total, g, std=60.0 if quant else 1.0)
        s["k_scale"], s["v_scale"] = (0.02, 0.015) if quant else (1.0, 1.0)
        s["q"] = normal(g, b, hq, d, std=2.0).to(dt)
        order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        table = torch.zeros((b, max(need)), dtype=torch.int32)
        begin = 0
        order = order.cpu()
        for i, n in enumerate(need):
            table[i, :n] = order[begin:begin + n]
            begin += n
        s["page_table"] = table.to(DEV)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.empty((b, hq, d), device=DEV, dtype=dt)
        s["lse"] = torch.empty((b, hq), device=DEV, dtype=torch.float32)
        s["status"] = torch.zeros(1, device=DEV, dtype=torch.int32)
        s["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)   # a program keeps one for all its calls
    else:
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // BLOCK), -(-n // BLOCK)
        f8 = torch.float8_e4m3fn
        a = torch.zeros((m, kb * BLOCK), device=DEV)
        a[:, :k] = normal(g, m, k) * torch.exp(normal(g, k, std=0.5))
        a = a.view(m, kb, BLOCK)
        s["a_scales"] = a.abs().amax(2).clamp(min=MIN_AMAX) / E4M3_MAX
        s["a"] = (a / s["a_scales"][:, :, None]).to(f8).view(m, kb * BLOCK)[:, :k].contiguous()
        b = torch.zeros((nb * BLOCK, kb * BLOCK), device=DEV)
        b[:n, :k] = normal(g, n, k, std=0.02)
        b = b.view(nb, BLOCK, kb, BLOCK)
        s["b_scales"] = b.abs().amax((1, 3)) / E4M3_MAX
        s["b"] = (b / s["b_scales"][:, None, :, None]).to(f8).view(nb * BLOCK, kb * BLOCK)[:n, :k].contiguous()
        s["out"] = torch.empty((m, n), device=DEV, dtype=dt)
        s["status"] = torch.zeros(1, device=DEV, dtype=torch.int32)
    return s


# ------------------------------------------------------------- the plain forms

def plain_quantize(y):
    """e4m3 values and scales of 32-bit rows, in groups of 128 columns (the last one may be shorter)."""
    n, h = y.shape
    groups = -(-h // BLOCK)
    wide = torch.zeros((n, groups * BLOCK), device=y.device)
    wide[:, :h] = y
    wide = wide.view(n, groups, BLOCK)
    amax = wide.abs().amax(2).clamp(min=MIN_AMAX)
    q = (wide * (E4M3_MAX / amax)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(n, groups * BLOCK)[:, :h], amax / E4M3_MAX


def plain_norm(s, case):
    r = s["x"].float()
    out = {}
    if case["residual"]:
        r = r + s["residual_in"].float()
        out["residual"] = r.to(s["x"].dtype)
    y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * s["weight"].float()
    if "y" in case["outputs"]:
        out["y"] = y.to(s["x"].dtype)
    if "q" in case["outputs"]:
        out["q"], out["scales"] = plain_quantize(y)
    return out


def plain_rotate(x, cos, sin, interleaved):
    """x in 32 bits [tokens][heads][dim]; cos, sin [tokens][rotary / 2]."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    rest = x[..., 2 * half:]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
    return torch.cat([turned, rest], 2)


def plain_append(s, case):
    half = case["rotary"] // 2
    row = s["cos_sin"][s["positions"].long()]
    cos, sin = row[:, :half], row[:, half:]
    q = plain_rotate(s["q_in"].float(), cos, sin, case["interleaved"])
    k = plain_rotate(s["k"].float(), cos, sin, case["interleaved"])
    v = s["v"].float()
    slots = s["slots"]
    if case["unused"]:
        used = slots >= 0
        k, v, slots = k[used], v[used], slots[used]
    page, at = slots // case["page"], slots % case["page"]
    if case["cache"] == "e4m3":
        k = (k * (1.0 / s["k_scale"])).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v * (1.0 / s["v_scale"])).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        s["k_cache"].view(torch.uint8)[page, at] = k
        s["v_cache"].view(torch.uint8)[page, at] = v
    else:
        s["k_cache"][page, at] = k.to(s["k_cache"].dtype)
        s["v_cache"][page, at] = v.to(s["v_cache"].dtype)
    return {"q": q.to(s["q_in"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def gather(cache, pages):
    """cache[pages]; 8-bit values are indexed as the bytes that they are."""
    return cache.view(torch.uint8)[pages].view(cache.dtype) if cache.dtype == torch.float8_e4m3fn else cache[pages]


def plain_attention(s, case):
    b, hq, hk, d = case["batch"], case["q_heads"], case["kv_heads"], case["dim"]
    table = s["page_table"].long()
    n = table.shape[1] * case["page"]

    def gathered(cache):
        return gather(cache, table).float().reshape(b, n, hk, d).permute(0, 2, 1, 3)

    q = s["q"].float().view(b, hk, hq // hk, d) * (s["scale"] * s["k_scale"])
    scores = q @ gathered(s["k_cache"]).transpose(2, 3)
    inside = torch.arange(n, device=DEV) < s["seq_lens"][:, None]
    scores = scores.masked_fill(~inside[:, None, None], -math.inf)
    top = scores.amax(3, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(3, keepdim=True)
    out = (p @ gathered(s["v_cache"])) * (s["v_scale"] / torch.where(total == 0, 1.0, total))
    lse = (top + torch.log(total)).view(b, hq)
    return {"out": out.reshape(b, hq, d).to(s["q"].dtype), "lse": lse}


def plain_gemm(s, case):
    k, n = case["k"], case["n"]
    a = s["a"].float() * s["a_scales"].repeat_interleave(BLOCK, 1)[:, :k]
    b = s["b"].float() * s["b_scales"].repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return {"out": (a @ b.t()).to(s["out"].dtype)}


PLAIN = {"norm": plain_norm, "quantize": lambda s, c: dict(zip(("q", "scales"), plain_quantize(s["x"].float()))),
         "append": plain_append, "attention": plain_attention, "gemm": plain_gemm}


# -------------------------------------------------------- the framework's calls

def own_norm(awq, s, case):
    awq.add_rmsnorm(s["x"], s["weight"], EPS, residual=s.get("residual_in"), residual_out=s.get("residual"), out=s.get("y"),
                    out_q=s.get("q"), out_scales=s.get("scales"))
    return {k: s[k] for k in ("residual", "y", "q", "scales") if k in s}


def own_quantize(awq, s, case):
    awq.quantize_fp8(s["x"], s["q"], s["scales"])
    return {"q": s["q"], "scales": s["scales"]}


def own_append(awq, s, case):
    awq.rope_append(s["q_in"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slots"], s["k_cache"], s["v_cache"], s["status"],
                    q_out=s["q"], interleaved=case["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"q": s["q"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def own_attention(awq, s, case):
    awq.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["seq_lens"], s["out"], s["workspace"], s["status"],
                        scale=s["scale"], lse=s["lse"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"out": s["out"], "lse": s["lse"]}


def own_gemm(awq, s, case):
    awq.fp8_gemm(s["a"], s["a_scales"], s["b"], s["b_scales"], s["out"], s["status"])
    return {"out": s["out"]}


OWN = {"norm": own_norm, "quantize": own_quantize, "append": own_append, "attention": own_attention, "gemm": own_gemm}


def run(state):
    case = state["case"]
    if own:
        import awq_int4_moe_gb300 as awq
        return OWN[case["op"]](awq, state, case)
    return PLAIN[case["op"]](state, case)


# ------------------------------------------------------- the definition, 64 bits

def exact_groups(y):
    """Unrounded 8-bit values and scales of 64-bit rows."""
    q, scales = torch.empty_like(y), []
    for c in range(0, y.shape[1], BLOCK):
        part = y[:, c:c + BLOCK]
        scale = part.abs().max(1, keepdim=True).values.clamp(min=MIN_AMAX) / E4M3_MAX
        q[:, c:c + BLOCK] = part / scale
        scales.append(scale)
    return q, torch.cat(scales, 1)


def exact_turn(x, angle_row, interleaved):
    half = angle_row.shape[1] // 2
    i = torch.arange(half, device=DEV)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    z = torch.complex(x[..., first], x[..., second]) * torch.complex(angle_row[:, :half], angle_row[:, half:])[:, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        q, scales = exact_groups(s["x"].double())
        return {"q": q, "scales": scales}
    if op == "norm":
        out = {}
        r = s["x"].double()
        if case["residual"]:
            r = r + s["residual_in"].double()
            out["residual"] = r
        y = r / torch.sqrt(torch.linalg.vector_norm(r, dim=1, keepdim=True) ** 2 / case["hidden"] + EPS) * s["weight"].double()
        if "y" in case["outputs"]:
            out["y"] = y
        if "q" in case["outputs"]:
            out["q"], out["scales"] = exact_groups(y)
        return out
    if op == "append":
        row = s["cos_sin"].double()[s["positions"].long()]
        out = {"q": exact_turn(s["q_in"].double(), row, case["interleaved"])}
        kept = case["tokens"] - case["unused"]
        for name, x, scale in (("k_cache", exact_turn(s["k"].double(), row, case["interleaved"]), s["k_scale"]),
                               ("v_cache", s["v"].double(), s["v_scale"])):
            flat = torch.zeros((s[name].shape[0] * case["page"], case["kv_heads"], case["dim"]), dtype=torch.float64, device=DEV)
            flat[s["slots"][:kept]] = (x / scale).clamp(-E4M3_MAX, E4M3_MAX)[:kept] if case["cache"] == "e4m3" else x[:kept]
            out[name] = flat.view(s[name].shape)
        return out
    if op == "attention":
        b, hq, hk, d = case["batch"], case["q_heads"], case["kv_heads"], case["dim"]
        out = torch.zeros((b, hq, d), dtype=torch.float64, device=DEV)
        lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device=DEV)
        for i, n in enumerate(lengths(case)):
            if n == 0:
                continue
            pages = s["page_table"][i, :pages_of(case, n)].long()
            for h in range(hk):
                k = gather(s["k_cache"][:, :, h], pages).double().reshape(-1, d)[:n] * s["k_scale"]
                v = gather(s["v_cache"][:, :, h], pages).double().reshape(-1, d)[:n] * s["v_scale"]
                group = slice(h * (hq // hk), (h + 1) * (hq // hk))
                score = s["q"][i, group].double() @ k.t() * s["scale"]
                lse[i, group] = torch.logsumexp(score, 1)
                out[i, group] = torch.softmax(score, 1) @ v
        return {"out": out, "lse": lse}
    m, n, k = case["m"], case["n"], case["k"]
    out = torch.zeros((m, n), dtype=torch.float64, device=DEV)
    for j, c in enumerate(range(0, k, BLOCK)):
        by_row = s["b_scales"][:, j].double().repeat_interleave(BLOCK)[:n]
        out += (s["a"][:, c:c + BLOCK].double() @ s["b"][:, c:c + BLOCK].double().t()) * s["a_scales"][:, j].double()[:, None] * by_row
    return {"out": out}
