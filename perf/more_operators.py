"""Further operators of the target's pass, in plain torch, with the cases they are timed on.

Around its matrix products a decoder with rotary positions that serves from a small cache needs

* ``rotate``  norms of each query and key head and their rotation by position, between the product
  that makes them and the cache;
* ``append``  the new tokens' keys and values into the pages of a cache held in 4 bits, and what
  then stands there, read back;
* ``attend``  the attention of the new tokens over that cache, causal, with an optional sliding
  window and a few first tokens that stay visible;
* ``score``   log-probabilities of given tokens, the entropy of each row and its likeliest ids.

The cache in 4 bits: 32 elements of a head share a power of two 2^e (the byte e + 127, 255 stands for
NaN), each element is a number of {0, 0.5, 1, 1.5, 2, 3, 4, 6} with a sign.  A page of a head holds
page x dim / 2 bytes of elements, row after row, two to a byte with the lower one in the low bits,
and then page x dim / 32 bytes of powers.

Where ``own`` is false, ``run`` computes the operators from elementary operations in 32 bits; where it
is true it calls the package.  Cases are dicts of plain values; lengths that differ between the
requests of a case follow from the case alone, values from the seed.
"""
import math

import torch

own = False

HEADS = {"32/8": (32, 8), "40/8": (40, 8), "8/2": (8, 2), "16/16": (16, 16), "64/8": (64, 8)}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _rotate_case(name, tokens, heads, dim, rotary, far, dtype, norm=True, interleaved=False):
    return {"name": name, "op": "rotate", "tokens": tokens, "heads": heads, "dim": dim, "rotary": rotary,
            "far": far, "dtype": dtype, "norm": norm, "interleaved": interleaved}


def _cache_case(name, op, batch, new, length, heads, dim, page, window=0, sinks=0):
    return {"name": name, "op": op, "batch": batch, "new": new, "length": length, "heads": heads,
            "dim": dim, "page": page, "window": window, "sinks": sinks}


def _score_case(name, rows, vocab, dtype, top, masked):
    return {"name": name, "op": "score", "rows": rows, "vocab": vocab, "dtype": dtype, "top": top,
            "masked": masked}


def listed():
    return [
        # one token of one chat far into its context: the latency of a launch
        _rotate_case("rotate_one_b1", 1, "32/8", 128, 128, 40000, "bf16"),
        # the 16 positions of 64 draft blocks
        _rotate_case("rotate_block_b64", 1024, "32/8", 128, 128, 9000, "bf16"),
        # a long prompt in one pass, 5 query heads to a key head (hidden width 5120)
        _rotate_case("rotate_prompt", 8191, "40/8", 128, 128, 8191, "bf16"),
        # the draft blocks of eight requests into the cache
        _cache_case("append_block_b8", "append", 8, 16, 4099, "32/8", 128, 16),
        # eight prompts, up to a thousand tokens each, laid into pages at once
        _cache_case("append_prompt_b8", "append", 8, 1024, 1024, "32/8", 128, 64),
        # the first tokens of a chat, one request: nothing but latency
        _cache_case("attend_one_b1_short", "attend", 1, 1, 37, "32/8", 128, 16),
        # eight requests check a whole draft block of 16 positions over medium contexts
        _cache_case("attend_block_b8", "attend", 8, 16, 4099, "32/8", 128, 16),
        # 64 requests decode one token each over long contexts: the cache's bytes
        _cache_case("attend_one_b64_long", "attend", 64, 1, 8192, "32/8", 128, 64),
        # two chunks of a prompt over what is already in the cache: matrix work
        _cache_case("attend_prompt_b2", "attend", 2, 2048, 5120, "32/8", 128, 64),
        # alternatives for the next token of one chat
        _score_case("score_one_b1", 1, 151936, "fp32", 20, False),
        # the rows of 64 draft blocks, every other one under a grammar, with alternatives
        _score_case("score_block_b64", 1024, 151936, "bf16", 5, True),
        # the probabilities of a prompt's own tokens
        _score_case("score_prompt", 777, 50257, "bf16", 0, False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "attend", "attend", "score"])
    if op == "rotate":
        dim = rng.choice([64, 128, 128, 256])
        case = _rotate_case("", _log_int(rng, 1, 4000), rng.choice(sorted(HEADS)), dim,
                            rng.choice([dim, dim, dim // 2, 48]), _log_int(rng, 1, 1_000_000),
                            rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.7, rng.random() < 0.3)
        del case["name"]
        if case["dtype"] == "fp32" or dim == 256:
            case["tokens"] = min(case["tokens"], 1500)
        return case
    if op in ("append", "attend"):
        case = {"op": op, "heads": rng.choice(sorted(HEADS)), "dim": rng.choice([64, 128, 128, 256]),
                "page": rng.choice([16, 32, 64, 128]), "window": 0, "sinks": 0}
        batch = _log_int(rng, 1, 64)
        kind = rng.choice(["one", "block", "prompt"])
        new = 1 if kind == "one" else rng.randint(2, 16) if kind == "block" else _log_int(rng, 17, 2048)
        if kind == "prompt":
            batch = max(1, min(batch, 4096 // new))
        # the cache of a case stays below that of the listed ones
        most = max(new, min(16384, 400_000 // batch // (2 if case["dim"] == 256 else 1)))
        if kind == "prompt":
            most = max(new, min(most, 5120))
        length = max(new, _log_int(rng, 1, most))
        if op == "attend" and rng.random() < 0.35:
            case["window"] = _log_int(rng, 1, 4096)
            case["sinks"] = rng.choice([0, 1, 4, 7, 64])
        case.update(batch=batch, new=new, length=length)
        return case
    case = _score_case("", _log_int(rng, 1, 1000), rng.choice([4096, 5003, 32000, 50257, 151936]),
                       rng.choice(["bf16", "fp32"]), rng.choice([0, 1, 5, 20, 64]), rng.random() < 0.4)
    del case["name"]
    if case["dtype"] == "fp32":
        case["rows"] = min(case["rows"], 400)
    return case


# ------------------------------------------------------------------ lengths of a case
def _spread(batch, lo, hi):
    """`batch` whole numbers in [lo, hi], the first of them hi."""
    return [hi if b == 0 else lo + (b * 2654435761 % (2 ** 32)) * (hi - lo + 1) // 2 ** 32
            for b in range(batch)]


def _lens(case):
    """New tokens and cache lengths (the new ones counted) of each request."""
    new = [case["new"]] * case["batch"] if case["new"] <= 16 else \
        _spread(case["batch"], (case["new"] + 1) // 2, case["new"])
    total = _spread(case["batch"], (case["length"] + 1) // 2, case["length"])
    return new, [max(n, t) for n, t in zip(new, total)]


def work(case):
    if case["op"] == "rotate":
        hq, hk = HEADS[case["heads"]]
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * (hq + hk) * case["dim"]
        return {"bytes": 2 * n * size + 4 * case["tokens"], "flops": 9 * n}
    if case["op"] == "score":
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["rows"] * case["vocab"]
        return {"bytes": n * size + case["rows"] * (12 + 8 * case["top"]), "flops": 7 * n}
    hq, hk = HEADS[case["heads"]]
    d = case["dim"]
    row = d // 2 + d // 32
    new, total = _lens(case)
    if case["op"] == "append":  # in, into the cache, and read from there in the type of the model
        return {"bytes": 2 * sum(new) * hk * (2 * d + row + row + 2 * d), "flops": 4 * sum(new) * hk * d}
    keys = pairs = 0
    w, s = case["window"], case["sinks"]
    for n, t in zip(new, total):
        if not w:
            keys += t
            pairs += n * t - n * (n - 1) // 2
            continue
        first = max(0, t - n - w + 1)
        keys += (t - first) + min(s, first)
        for i in range(n):
            p = t - n + i
            lo = max(0, p - w + 1)
            pairs += p - lo + 1 + min(s, lo)
    return {"bytes": 2 * keys * hk * row + 4 * sum(new) * hq * d + 4 * sum(new) * hq, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ inputs
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _rotate_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq, hk = HEADS[case["heads"]]
    d, dt, n = case["dim"], TYPES[case["dtype"]], case["tokens"]
    # queries, keys and values as one product leaves them, some channels larger than others
    qkv = torch.randn((n, hq + 2 * hk, d), generator=g, device="cuda")
    qkv *= torch.rand((hq + 2 * hk, d), generator=g, device="cuda") * 2 + 0.5
    q, k, _ = qkv.to(dt).split([hq, hk, hk], 1)
    # a few runs of consecutive positions, as requests bring them
    runs = min(n, 1 + n // 500 if n > 16 else 1)
    first = torch.randint(0, max(1, case["far"] - n // runs), (runs,), generator=g, device="cuda")
    at = torch.arange(n, device="cuda")
    state = {"case": case, "q": q, "k": k, "positions": (first[at * runs // n] + at % (-(-n // runs))).to(torch.int32),
             "q_weight": None, "k_weight": None,
             "inv_freq": 1e6 ** (-torch.arange(0, case["rotary"], 2, dtype=torch.float64) / case["rotary"])}
    if case["norm"]:
        for name in ("q_weight", "k_weight"):
            state[name] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
    return state


def _powers(x):
    """Exponents of the blocks of 32 of x [..., dim]: the least with max |x| <= 7 * 2^e, [..., dim / 32]."""
    part, e = torch.frexp(x.unflatten(-1, (-1, 32)).abs().amax(-1))
    return torch.where(part == 0, -125, e - 3 + (part > 0.875).int()).clamp(-125, 125)


def _steps(x, e):
    """x in units of 2^e, rounded to the numbers that 4 bits hold: nearest, ties to the even code."""
    y = torch.ldexp(x.unflatten(-1, (-1, 32)), -e[..., None])
    size = y.abs()
    step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0))
    return torch.copysign(((size / step).round() * step).clamp(max=6.0), y)


def _encode(x):
    """Rows x [..., rows, dim] as a page of a head holds them: [..., rows * (dim / 2 + dim / 32)] bytes."""
    e = _powers(x)
    y = _steps(x, e).flatten(-2)
    size = y.abs()
    code = torch.where(size < 2, size * 2, torch.where(size < 4, size + 2, size / 2 + 4)).to(torch.uint8)
    code += (torch.signbit(y).to(torch.uint8) << 3)
    code = code[..., 0::2] | (code[..., 1::2] << 4)
    return torch.cat([code.flatten(-2), (e + 127).to(torch.uint8).flatten(-2)], -1)


def _cache_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq, hk = HEADS[case["heads"]]
    d, ps = case["dim"], case["page"]
    new, total = _lens(case)
    tokens = sum(new)
    pages = [-(-t // ps) for t in total]
    num, width = sum(pages) + 3, max(pages)
    page_bytes = ps * (d // 2 + d // 32)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    def cache():
        # what earlier tokens left: rows as a projection gives them, some channels larger than others
        size = torch.rand((hk, 1, d), generator=g, device="cuda") + 0.5
        out = torch.empty((num, hk, page_bytes), dtype=torch.uint8, device="cuda")
        step = max(1, 2 ** 26 // (hk * ps * d))
        for i in range(0, num, step):
            n = min(step, num - i)
            out[i:i + n] = _encode(torch.randn((n, hk, ps, d), generator=g, device="cuda") * size)
        return out

    order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    owned = torch.arange(width, device="cuda")[None] < torch.tensor(pages, device="cuda")[:, None]
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device="cuda")
    table[owned] = order[:sum(pages)]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    state = {"case": case, "k_cache": cache(), "v_cache": cache(), "page_table": table,
             "kv_len": _ints(total), "q_start": _ints(starts), "max_new": max(new), "max_kv": max(total)}
    if case["op"] == "append":
        state.update(k=normal(tokens, hk, d), v=normal(tokens, hk, d))
    else:
        state.update(q=normal(tokens, hq, d))
    return state


def _score_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, v = case["rows"], case["vocab"]
    logits = torch.randn((n, v), generator=g, device="cuda").mul_(2.5)
    # the text mostly says what the model would have said
    tokens = (torch.rand(n, generator=g, device="cuda") ** 3 * v).long().clamp_(max=v - 1)
    likely = torch.rand(n, generator=g, device="cuda") < 0.7
    logits.scatter_add_(1, tokens[:, None], torch.where(likely, 14.0, 3.0)[:, None])
    if case["masked"]:
        hide = torch.rand((n, v), generator=g, device="cuda") < 0.5
        hide[0::2] = False
        hide.scatter_(1, tokens[:, None], False)
        logits.masked_fill_(hide, -math.inf)
    tokens = tokens.to(torch.int32)
    tokens[7::16] = -1  # rows of a padded batch
    return {"case": case, "logits": logits.to(TYPES[case["dtype"]]), "tokens": tokens}


def _inputs(case, seed):
    if case["op"] == "rotate":
        return _rotate_inputs(case, seed)
    return _score_inputs(case, seed) if case["op"] == "score" else _cache_inputs(case, seed)


def prepare(case, seed):
    state = _inputs(case, seed)
    if own:
        from gru_corrected_draft_amd import verify
        if case["op"] == "rotate":
            hq, hk = HEADS[case["heads"]]
            state["rotation"] = verify.HeadRotation(hq, hk, case["dim"], state["inv_freq"], TYPES[case["dtype"]],
                                                    interleaved=case["interleaved"])
        elif case["op"] == "score":
            state["scores"] = verify.TokenScores(case["vocab"], TYPES[case["dtype"]], max_rows=case["rows"])
        else:
            hq, hk = HEADS[case["heads"]]
            state["attention"] = verify.PagedAttention4(hq, hk, case["dim"], case["page"], max_requests=case["batch"])
    elif case["op"] == "rotate":
        state["inv_freq"] = state["inv_freq"].cuda()
    elif case["op"] != "score":
        # the numbers of a byte's two codes
        grid = torch.tensor(GRID + tuple(-x for x in GRID), device="cuda")
        byte = torch.arange(256, device="cuda")
        state["pairs"] = torch.stack([grid[byte % 16], grid[byte // 16]], 1)
    return state


# ------------------------------------------------------------------ plain forms
def _plain_rotate(s):
    case = s["case"]
    r = case["rotary"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        if case["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s[name + "_weight"].float()
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if case["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
        turned = [a * cos - b * sin, b * cos + a * sin]
        turned = torch.stack(turned, -1).flatten(-2) if case["interleaved"] else torch.cat(turned, -1)
        out[name] = torch.cat([turned, x[..., r:]], -1).to(s[name].dtype)
    return out


def _token_owner(s):
    """Request and cache position of each new token."""
    start, kv = s["q_start"].long(), s["kv_len"].long()
    at = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(start[1:], at, right=True)
    return b, kv[b] - (start[b + 1] - at)


def _row_places(s, pos):
    """First byte of the elements and of the powers of the rows at ``pos`` in their pages."""
    d, ps = s["case"]["dim"], s["case"]["page"]
    row = pos % ps
    return row * (d // 2), ps * (d // 2) + row * (d // 32)


def _rows_of(s, cache, page, pos):
    """Rows of the cache in 32 bits: [..., kv_heads, dim] for pages and positions [...]."""
    d = s["case"]["dim"]
    heads = torch.arange(cache.shape[1], device="cuda")[:, None]
    data, power = _row_places(s, pos)
    page = page[..., None, None]
    x = cache[page, heads, data[..., None, None] + torch.arange(d // 2, device="cuda")]
    e = cache[page, heads, power[..., None, None] + torch.arange(d // 32, device="cuda")].int()
    two = torch.ldexp(torch.ones((), device="cuda"), e - 127)
    two = torch.where(e == 255, math.nan, two)
    return (s["pairs"][x.int()].flatten(-2).unflatten(-1, (-1, 32)) * two[..., None]).flatten(-2)


def _plain_append(s):
    ps, d = s["case"]["page"], s["case"]["dim"]
    b, pos = _token_owner(s)
    page = s["page_table"].long()[b, pos // ps]
    data, power = _row_places(s, pos)
    out = {}
    for name in ("k", "v"):
        cache = s[name + "_cache"]
        heads = torch.arange(cache.shape[1], device="cuda")[:, None]
        row = _encode(s[name].float()[:, :, None])
        at = page[:, None, None]
        cache[at, heads, data[:, None, None] + torch.arange(d // 2, device="cuda")] = row[..., :d // 2]
        cache[at, heads, power[:, None, None] + torch.arange(d // 32, device="cuda")] = row[..., d // 2:]
        out[name] = _rows_of(s, cache, page, pos).to(torch.bfloat16)
    return out


def _plain_attend(s):
    case = s["case"]
    hq, hk = HEADS[case["heads"]]
    d, ps, w, sinks = case["dim"], case["page"], case["window"], case["sinks"]
    batch, n = case["batch"], s["max_new"]
    start, kv = s["q_start"].long(), s["kv_len"].long()
    new = start[1:] - start[:-1]
    if w and w + n - 1 + sinks < s["max_kv"]:  # only what a window can reach is gathered
        lo = (kv - new - w + 1).clamp(min=0)
        pos = torch.cat([torch.arange(sinks, device="cuda").expand(batch, sinks),
                         lo[:, None] + torch.arange(w + n - 1, device="cuda")], 1)
        once = torch.ones_like(pos, dtype=torch.bool)
        once[:, :sinks] = pos[:, :sinks] < lo[:, None]
    else:
        pos = torch.arange(s["max_kv"], device="cuda").expand(batch, -1)
        once = torch.ones_like(pos, dtype=torch.bool)
    there = once & (pos < kv[:, None])
    safe = pos.minimum(kv[:, None] - 1)
    page = s["page_table"].long().gather(1, safe // ps).clamp(min=0)
    k = _rows_of(s, s["k_cache"], page, safe)  # [batch, keys, hk, d]
    v = _rows_of(s, s["v_cache"], page, safe)
    # the new tokens of each request side by side, rows past its own repeated
    step = torch.arange(n, device="cuda")
    token = (start[:-1, None] + step.minimum(new[:, None] - 1))
    q = s["q"][token].float().view(batch, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(batch, hk, -1, d)
    score = (q @ k.permute(0, 2, 3, 1).contiguous()).view(batch, hk, hq // hk, n, -1).mul_(1.0 / math.sqrt(d))
    qpos = (kv - new)[:, None] + step
    seen = there[:, None] & (pos[:, None] <= qpos[:, :, None])
    if w:
        seen &= (pos[:, None] > qpos[:, :, None] - w) | (pos[:, None] < sinks)
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(batch, hk, -1, p.shape[-1]) @ v.permute(0, 2, 1, 3).contiguous()).view(batch, hk, hq // hk, n, d)
    out = out / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    real = step < new[:, None]
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(batch, n, hq, d)[real].to(s["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(batch, n, hq)[real]}


def _plain_score(s):
    case = s["case"]
    x = s["logits"].float()
    m = x.amax(1, keepdim=True)
    y = x - m
    e = y.exp()
    total = e.sum(1)
    norm = total.log()
    entropy = norm - torch.where(e > 0, e * y, 0.0).sum(1) / total
    tokens = s["tokens"].long()
    logprob = y.gather(1, tokens.clamp(min=0)[:, None]).squeeze(1) - norm
    out = {"logprob": logprob.masked_fill(tokens < 0, -math.inf), "entropy": entropy}
    if case["top"]:
        # one whole number for each logit that orders them, the lower id first among equal ones
        bits = (x + 0.0).view(torch.int32).long()
        bits = torch.where(bits < 0, -2 ** 31 - bits, bits)
        ids = (bits * 2 ** 32 + (2 ** 32 - 1 - torch.arange(case["vocab"], device="cuda"))).topk(case["top"], 1)[1]
        out.update(ids=ids.int(), values=y.gather(1, ids) - norm[:, None])
    return out


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"rotate": _plain_rotate, "append": _plain_append, "attend": _plain_attend, "score": _plain_score}[op](s)
    if op == "rotate":
        q, k = s["rotation"].run(s["q"], s["k"], s["positions"], s["q_weight"], s["k_weight"], eps=EPS)
        return {"q": q, "k": k}
    if op == "score":
        logprob, entropy, ids, values = s["scores"].run(s["logits"], s["tokens"], top=case["top"])
        out = {"logprob": logprob, "entropy": entropy}
        if case["top"]:
            out.update(ids=ids, values=values)
        return out
    where = (s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"], s["q_start"])
    if op == "append":
        s["attention"].append(s["k"], s["v"], *where, max_new=s["max_new"])
        k, v = s["attention"].read(s["k"].shape[0], *where, max_new=s["max_new"])
        return {"k": k, "v": v}
    out, lse = s["attention"].run(s["q"], *where, max_new=s["max_new"], max_kv=s["max_kv"],
                                  window=case["window"], sinks=case["sinks"], return_lse=True)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ 64 bits, from the definitions
def _exact_rotate(s):
    case = s["case"]
    r = case["rotary"]
    freq = torch.tensor([1e6 ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64, device="cuda")
    angle = s["positions"].double()[:, None] * freq
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        if case["norm"]:
            x = x / ((x ** 2).sum(-1, keepdim=True) / case["dim"] + EPS).sqrt()
            x = x * s[name + "_weight"].double()
        y = x.clone()
        if case["interleaved"]:
            y[..., :r] = torch.view_as_real(torch.view_as_complex(x[..., :r].unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
        else:
            z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
            y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
        out[name] = y
    return out


def _exact_append(s):
    """Each number by the nearest of the sixteen, blocks one power of two after the other."""
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
    out = {}
    for name in ("k", "v"):
        x = s[name].double().unflatten(-1, (-1, 32))
        top = x.abs().amax(-1, keepdim=True)
        unit = torch.full_like(top, 2.0 ** -125)
        for e in range(-124, 126):
            unit = torch.where(top > 7 * unit, 2.0 ** e, unit)
        y = (x.abs() / unit).clamp(max=6.0)
        far = (y[..., None] - grid).abs()
        near = far.amin(-1, keepdim=True)
        code = torch.arange(8, device="cuda")
        # among the nearest ones the even code
        pick = torch.where(far == near, torch.where(code % 2 == 0, 2, 1), 0).argmax(-1)
        out[name] = (grid[pick] * unit * torch.sign(x)).flatten(-2)
    return out


def _exact_attend(s):
    case = s["case"]
    hq, hk = HEADS[case["heads"]]
    w, d, ps = case["window"], case["dim"], case["page"]
    start, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    grid = torch.tensor(GRID + tuple(-x for x in GRID), dtype=torch.float64, device="cuda")

    def rows(cache, pages, h, n):
        raw = cache[pages, h]
        data = raw[:, :ps * d // 2].reshape(-1, d // 2)[:n].int()
        power = raw[:, ps * d // 2:].reshape(-1, d // 32)[:n].double() - 127
        x = torch.stack([grid[data & 15], grid[data >> 4]], -1).reshape(n, -1, 32)
        return (x * torch.exp2(power)[..., None]).reshape(n, d)

    outs, lses = [], []
    for b, n in enumerate(lens):
        pages = s["page_table"][b, :-(-n // ps)].long()
        q = s["q"][start[b]:start[b + 1]].double()
        place = torch.arange(n, device="cuda")
        mine = torch.arange(n - q.shape[0], n, device="cuda")[:, None]
        hidden = place > mine
        if w:
            hidden |= (mine - place >= w) & (place >= case["sinks"])
        out, lse = torch.empty_like(q), q.new_empty(q.shape[:2])
        for kh in range(hk):
            keys, values = rows(s["k_cache"], pages, kh, n), rows(s["v_cache"], pages, kh, n)
            for h in range(kh * hq // hk, (kh + 1) * hq // hk):
                a = (torch.mm(q[:, h], keys.t().contiguous()) / d ** 0.5).masked_fill(hidden, -math.inf)
                lse[:, h] = torch.logsumexp(a, 1)
                out[:, h] = torch.mm(torch.softmax(a, 1), values)
        outs.append(out)
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_score(s):
    case = s["case"]
    rows = {"logprob": [], "entropy": [], "ids": [], "values": []}
    for x, token in zip(s["logits"], s["tokens"].tolist()):
        p = torch.log_softmax(x.double(), 0)
        rows["logprob"].append(p[token] if token >= 0 else p.new_tensor(-math.inf))
        rows["entropy"].append(-torch.special.xlogy(p.exp(), p.exp()).sum())
        if case["top"]:
            ids = torch.sort(x.double(), descending=True, stable=True)[1][:case["top"]]
            rows["ids"].append(ids.int())
            rows["values"].append(p[ids])
    return {name: torch.stack(r) for name, r in rows.items() if r}


def exact(case, seed):
    s = _inputs(case, seed)
    return {"rotate": _exact_rotate, "append": _exact_append, "attend": _exact_attend, "score": _exact_score}[case["op"]](s)
