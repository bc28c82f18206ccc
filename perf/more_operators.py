"""Work of the prompt's operators of the decoder layer: causal attention over
packed prompts, attention of a chunk of new tokens over the paged cache, and
the norm of each head of q and k with the rotation and the append to that cache.

Each case is a dict of plain values. ``run`` computes the operator in its
plain form (elementary torch operations in 32 bits, rounded once), or, where
``own`` is true, through the framework's public calls on the same inputs.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f16": 2, "bf16": 2, "e4m3": 1}


# ------------------------------------------------------------------- the cases

def prompt(name, lens, behind, q_heads, kv_heads, dim, dtype):
    """lens: the sequences' lengths, as text; behind: rows of the buffers past the last sequence."""
    return {"name": name, "op": "prompt", "lens": lens, "behind": behind, "q_heads": q_heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype}


def chunk(name, lens, news, q_heads, kv_heads, dim, dtype, cache, page, heads_first):
    """lens: tokens of each sequence in the cache, its new ones among them; news: how many of them are new."""
    return {"name": name, "op": "chunk", "lens": lens, "news": news, "behind": 0, "q_heads": q_heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "cache": cache, "page": page, "heads_first": heads_first}


def append(name, tokens, unused, q_heads, kv_heads, dim, rotary, interleaved, dtype, cache, page, heads_first):
    return {"name": name, "op": "append", "tokens": tokens, "unused": unused, "q_heads": q_heads, "kv_heads": kv_heads,
            "dim": dim, "rotary": rotary, "interleaved": interleaved, "dtype": dtype, "cache": cache, "page": page,
            "heads_first": heads_first}


def spread(n, most, first):
    """n lengths from 1 to `most`, spread over the range; the first is `first`."""
    return [first] + [max(1, int(most * ((i * 0.6180339887498949) % 1.0))) for i in range(1, n)]


def text(values):
    return " ".join(str(v) for v in values)


def numbers(words):
    return [int(w) for w in words.split()]


def listed():
    return [
        # one short question, heads of the example's layer: latency
        prompt("prompt_b1_len48", "48", 0, 20, 4, 128, "f16"),
        # a batch of prompts packed one behind the other, an empty one among them, the buffer's end unused
        prompt("prompt_b13_ragged", text(spread(12, 2000, 1999) + [0]), 37, 32, 8, 128, "bf16"),
        # a long prompt
        prompt("prompt_b1_len8192", "8192", 0, 32, 8, 128, "bf16"),
        # prompts of a model with wide heads
        prompt("prompt_b4_dim256", "3001 1024 2500 777", 0, 16, 2, 256, "f16"),
        # many short prompts of a model with small heads, as many KV heads as query heads
        prompt("prompt_b40_dim64", text(spread(40, 700, 650)), 0, 16, 16, 64, "f16"),
        # one user's five drafted tokens, short context: latency
        chunk("chunk_b1_new5_len700", "700", "5", 20, 4, 128, "f16", "f16", 16, False),
        # four drafted tokens of each sequence of a serving batch, 8-bit cache
        chunk("chunk_b32_new4_e4m3", text(spread(32, 16000, 16000)), text([4] * 32), 64, 8, 128, "bf16", "e4m3", 64, True),
        # the next 1024 tokens of a prompt of which most is in the cache
        chunk("chunk_b1_new1024_len32768", "32768", "1024", 32, 4, 128, "bf16", "bf16", 32, False),
        # a step that mixes chunks of prompts with sequences that decode one token, 8-bit cache
        chunk("chunk_b19_mixed_e4m3", text([5000, 2048, 1500] + spread(16, 9000, 8000)), text([1000, 2048, 333] + [1] * 16),
              20, 4, 128, "f16", "e4m3", 16, False),
        # one decode step of a padded batch, q/k/v cut from the QKV product
        append("append_decode16", 16, 2, 20, 4, 128, 128, False, "f16", "f16", 16, False),
        # a long prompt into an 8-bit cache, heads before tokens in a page
        append("append_prompt8191", 8191, 0, 32, 8, 128, 128, False, "bf16", "e4m3", 64, True),
        # a batch of prompts, pairs interleaved, a part of the head rotated
        append("append_prompt2500_partial", 2500, 0, 16, 2, 256, 64, True, "f16", "f16", 24, False),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_FLOPS = 4.0 * 8192 * 8193 / 2 * 32 * 128     # of the long prompt
MOST_BYTES = 5.0e8                                # of the serving batch's cache


def draw(rng):
    op = rng.choice(["prompt", "prompt", "chunk", "chunk", "append"])
    dtype = rng.choice(["f16", "bf16"])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 5, 7, 8, 16])
    dim = rng.choice([64, 80, 96, 128, 128, 256])
    cache, page, first = rng.choice([dtype, "e4m3"]), rng.choice([1, 16, 24, 64, 256]), rng.random() < 0.5
    if op == "append":
        tokens = log_int(rng, 1, max(1, min(16384, 8191 * 48 * 128 // ((heads + 2 * kv) * dim))))
        case = append("", tokens, rng.choice([0, 0, tokens // 8]), heads, kv, dim, rng.choice([dim, dim, dim // 2]),
                      rng.random() < 0.3, dtype, cache, page, first)
        del case["name"]
        return case
    batch = log_int(rng, 1, 48)
    if op == "prompt":
        most = min(math.sqrt(MOST_FLOPS / (2.0 * heads * dim * batch)), MOST_BYTES / (4.0 * (heads + kv) * dim * batch))
        lens = spread(batch, *2 * [log_int(rng, 1, max(1, min(8192, int(most))))])
        if batch > 2 and rng.random() < 0.3:
            lens[rng.randrange(1, batch)] = 0
        case = prompt("", text(lens), rng.choice([0, 0, 17]), heads, kv, dim, dtype)
    else:
        news = log_int(rng, 1, 2048)
        longest = min(MOST_FLOPS / (4.0 * heads * dim * batch * news), MOST_BYTES / (4.0 * kv * dim * batch), 131072)
        lens = spread(batch, *2 * [log_int(rng, 1, max(1, int(longest)))])
        some = [min(n, news if rng.random() < 0.6 else rng.choice([1, 1, max(1, news // 3)])) for n in lens]
        case = chunk("", text(lens), text(some), heads, kv, dim, dtype, cache, page, first)
    del case["name"]
    return case


def sequences(case):
    """Of each sequence: its first row, its new tokens, all its tokens."""
    lens = numbers(case["lens"])
    news = numbers(case["news"]) if case["op"] == "chunk" else lens
    out, at = [], 0
    for n, new in zip(lens, news):
        out.append((at, new, n))
        at += new
    return out


def work(case):
    w, d = SIZE[case["dtype"]], case["dim"]
    hq, hk = case["q_heads"], case["kv_heads"]
    if case["op"] == "append":
        t, kept = case["tokens"], case["tokens"] - case["unused"]
        b = t * hq * d * 2 * w + kept * hk * d * 2 * (w + SIZE[case["cache"]]) + t * (case["rotary"] * 4 + 12) + 2 * d * w
        return {"bytes": b, "flops": (t * hq + kept * hk) * (3 * case["rotary"] + 4 * d)}
    seqs = sequences(case)
    rows = sum(new for _, new, _ in seqs)
    kept = sum(n for _, _, n in seqs)
    pairs = sum(new * n - new * (new - 1) // 2 for _, new, n in seqs)
    kv = SIZE[case["cache"]] if case["op"] == "chunk" else w
    return {"bytes": rows * hq * (2 * d * w + 4) + 2 * kept * hk * d * kv, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ the inputs

def normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std


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
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    s["status"] = torch.zeros(1, device=DEV, dtype=torch.int32)
    if case["op"] == "append":
        t = case["tokens"]
        # channels of different size, as a projection gives them before the norm
        qkv = (normal(g, t, hq + 2 * hk, d, std=3.0) * torch.exp(normal(g, hq + 2 * hk, d, std=0.5))).to(dt)
        s["q_in"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["q_weight"], s["k_weight"] = (1.0 + normal(g, d, std=0.2)).to(dt), (1.0 + normal(g, d, std=0.2)).to(dt)
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
        s["k_scale"], s["v_scale"] = (0.02, 0.05) if case["cache"] == "e4m3" else (1.0, 1.0)
        return s
    seqs = sequences(case)
    rows = sum(new for _, new, _ in seqs) + case["behind"]
    s["cu_seqlens"] = torch.tensor([at for at, _, _ in seqs] + [rows - case["behind"]], dtype=torch.int32, device=DEV)
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.zeros((rows, hq, d), device=DEV, dtype=dt)
    s["lse"] = torch.zeros((rows, hq), device=DEV, dtype=torch.float32)
    s["workspace"] = torch.zeros(96 << 20, dtype=torch.uint8, device=DEV)   # a program keeps one for all its calls
    if case["op"] == "prompt":
        # q, k and v as they come out of one product, q larger (its weights are)
        qkv = normal(g, rows, hq + 2 * hk, d)
        qkv[:, :hq] *= 2.0
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        return s
    quant = case["cache"] == "e4m3"
    need = [pages_of(case, n) for _, _, n in seqs]
    total = sum(need) + 1
    s["k_cache"] = cache_of(case, total, g, std=50.0 if quant else 1.0)
    s["v_cache"] = cache_of(case, total, g, std=60.0 if quant else 1.0)
    s["k_scale"], s["v_scale"] = (0.02, 0.015) if quant else (1.0, 1.0)
    s["q"] = normal(g, rows, hq, d, std=2.0).to(dt)
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.zeros((len(need), max(need)), dtype=torch.int32)
    begin = 0
    for i, n in enumerate(need):
        table[i, :n] = order[begin:begin + n]
        begin += n
    s["page_table"] = table.to(DEV)
    s["seq_lens"] = torch.tensor([n for _, _, n in seqs], dtype=torch.int32, device=DEV)
    return s


def gather(cache, pages):
    """cache[pages]; 8-bit values are indexed as the bytes that they are."""
    return cache.view(torch.uint8)[pages].view(cache.dtype) if cache.dtype == torch.float8_e4m3fn else cache[pages]


# ------------------------------------------------------------- the plain forms

def plain_rows(q, k, v, first, scale, v_scale):
    """Attention of q [rows][heads][dim], whose row i sees the first `first + i` of k, v [tokens][KV heads][dim]."""
    rows, hq, d = q.shape
    n, hk, _ = k.shape
    q = (q.float() * scale).view(rows, hk, hq // hk, d).permute(1, 2, 0, 3)
    scores = q @ k.float().permute(1, 2, 0)[:, None]
    seen = torch.arange(n, device=DEV) < first + torch.arange(rows, device=DEV)[:, None]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(3, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(3, keepdim=True)
    out = (p @ v.float().permute(1, 0, 2)[:, None]) * (v_scale / total)
    lse = (top + torch.log(total))[..., 0]
    return out.permute(2, 0, 1, 3).reshape(rows, hq, d), lse.permute(2, 0, 1).reshape(rows, hq)


def plain_attention(s, case):
    for b, (at, new, n) in enumerate(sequences(case)):
        if new == 0:
            continue
        if case["op"] == "prompt":
            k, v, k_scale, v_scale = s["k"][at:at + n], s["v"][at:at + n], 1.0, 1.0
        else:
            pages = s["page_table"][b, :pages_of(case, n)].long()
            k, v = (gather(c, pages).flatten(0, 1)[:n] for c in (s["k_cache"], s["v_cache"]))
            k_scale, v_scale = s["k_scale"], s["v_scale"]
        out, lse = plain_rows(s["q"][at:at + new], k, v, n - new + 1, s["scale"] * k_scale, v_scale)
        s["out"][at:at + new] = out.to(s["out"].dtype)
        s["lse"][at:at + new] = lse
    return {"out": s["out"], "lse": s["lse"]}


def plain_norm(x, weight):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) * weight.float()


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
    q = plain_rotate(plain_norm(s["q_in"], s["q_weight"]), cos, sin, case["interleaved"])
    k = plain_rotate(plain_norm(s["k"], s["k_weight"]), cos, sin, case["interleaved"])
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


PLAIN = {"prompt": plain_attention, "chunk": plain_attention, "append": plain_append}


# -------------------------------------------------------- the framework's calls

def own_prompt(awq, s, case):
    awq.prompt_attention(s["q"], s["k"], s["v"], s["cu_seqlens"], s["out"], s["workspace"], s["status"], scale=s["scale"],
                         lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def own_chunk(awq, s, case):
    awq.chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["cu_seqlens"], s["seq_lens"], s["out"],
                        s["workspace"], s["status"], scale=s["scale"], lse=s["lse"], k_scale=s["k_scale"],
                        v_scale=s["v_scale"])
    return {"out": s["out"], "lse": s["lse"]}


def own_append(awq, s, case):
    awq.qk_norm_rope_append(s["q_in"], s["k"], s["v"], s["q_weight"], s["k_weight"], EPS, s["positions"], s["cos_sin"],
                            s["slots"], s["k_cache"], s["v_cache"], s["status"], q_out=s["q"],
                            interleaved=case["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"q": s["q"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


OWN = {"prompt": own_prompt, "chunk": own_chunk, "append": own_append}


def run(state):
    case = state["case"]
    if own:
        import awq_int4_moe_gb300 as awq
        return OWN[case["op"]](awq, state, case)
    return PLAIN[case["op"]](state, case)


# ------------------------------------------------------- the definition, 64 bits

def exact_head(x, weight):
    x = x.double()
    return x / torch.sqrt(torch.linalg.vector_norm(x, dim=2, keepdim=True) ** 2 / x.shape[2] + EPS) * weight.double()


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
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        row = s["cos_sin"].double()[s["positions"].long()]
        turned = exact_turn(exact_head(s["k"], s["k_weight"]), row, case["interleaved"])
        out = {"q": exact_turn(exact_head(s["q_in"], s["q_weight"]), row, case["interleaved"])}
        kept = case["tokens"] - case["unused"]
        for name, x, scale in (("k_cache", turned, s["k_scale"]), ("v_cache", s["v"].double(), s["v_scale"])):
            flat = torch.zeros((s[name].shape[0] * case["page"], hk, d), dtype=torch.float64, device=DEV)
            flat[s["slots"][:kept]] = (x / scale).clamp(-E4M3_MAX, E4M3_MAX)[:kept] if case["cache"] == "e4m3" else x[:kept]
            out[name] = flat.view(s[name].shape)
        return out
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    for b, (at, new, n) in enumerate(sequences(case)):
        if new == 0:
            continue
        hidden = torch.ones((new, n), dtype=torch.bool, device=DEV).triu(n - new + 1)
        for h in range(hk):
            if case["op"] == "prompt":
                k, v = s["k"][at:at + n, h].double(), s["v"][at:at + n, h].double()
            else:
                pages = s["page_table"][b, :pages_of(case, n)].long()
                k = gather(s["k_cache"][:, :, h], pages).double().reshape(-1, d)[:n] * s["k_scale"]
                v = gather(s["v_cache"][:, :, h], pages).double().reshape(-1, d)[:n] * s["v_scale"]
            for i in range(h * (hq // hk), (h + 1) * (hq // hk)):
                score = (s["q"][at:at + new, i].double() @ k.t() * s["scale"]).masked_fill_(hidden, -math.inf)
                lse[at:at + new, i] = torch.logsumexp(score, 1)
                out[at:at + new, i] = torch.softmax(score, 1) @ v
    return {"out": out, "lse": lse}
