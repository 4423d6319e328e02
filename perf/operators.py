"""The operators that follow a draft block, in plain torch, with the cases they are timed on.

A rollout proposes up to 15 tokens for each request; the target model then scores the block in
one pass.  Four operators carry that pass around the target's own matrix products:

* ``append``  writes the block's keys and values into the pages of a key-value cache;
* ``attend``  is the attention of the new tokens over their request's pages, causal, with an
  optional sliding window and a few first tokens that stay visible;
* ``process`` applies repetition, frequency and presence penalties, biases and grammar masks to
  the target's logits, where row t of a request has also seen the proposals before it;
* ``verify``  decides from the processed logits how many proposals stand and which token follows.

Where ``own`` is false, ``run`` computes them from elementary operations in 32 bits; where it is
true it calls the package.  Cases are dicts of plain values; lengths that differ between the
requests of a case follow from the case alone, values from the seed.
"""
import math

import torch

own = False

HEADS = {"32/8": (32, 8), "40/8": (40, 8), "8/2": (8, 2), "16/16": (16, 16), "64/8": (64, 8)}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _cache_case(name, op, batch, new, length, heads, dim, page, dtype, window=0, sinks=0):
    return {"name": name, "op": op, "batch": batch, "new": new, "length": length, "heads": heads,
            "dim": dim, "page": page, "dtype": dtype, "window": window, "sinks": sinks}


def _logits_case(name, op, batch, rows, vocab, dtype, history, bias, mask, temperature=0.0):
    return {"name": name, "op": op, "batch": batch, "rows": rows, "vocab": vocab, "dtype": dtype,
            "history": history, "bias": bias, "mask": mask, "temperature": temperature}


def listed():
    return [
        # one token of one request into its cache: the latency of a launch
        _cache_case("append_one_b1", "append", 1, 1, 500, "32/8", 128, 16, "bf16"),
        # eight prompts, up to a thousand tokens each, laid into pages at once
        _cache_case("append_prompt_b8", "append", 8, 1024, 1024, "32/8", 128, 64, "bf16"),
        # the first tokens of a chat, one request: nothing but latency
        _cache_case("attend_one_b1_short", "attend", 1, 1, 37, "32/8", 128, 16, "bf16"),
        # eight requests check a whole draft block of 16 positions over medium contexts
        _cache_case("attend_block_b8", "attend", 8, 16, 4099, "32/8", 128, 16, "bf16"),
        # 64 requests decode one token each over long contexts: the cache's bytes
        _cache_case("attend_one_b64_long", "attend", 64, 1, 8192, "32/8", 128, 64, "bf16"),
        # a draft block over a very long context in a layer with a window and four sinks; 5 query
        # heads share a key head (hidden width 5120)
        _cache_case("attend_window_b16", "attend", 16, 16, 32000, "40/8", 128, 64, "bf16", 4096, 4),
        # two chunks of a prompt over what is already in the cache: matrix work
        _cache_case("attend_prompt_b2", "attend", 2, 2048, 5120, "32/8", 128, 64, "bf16"),
        # a small fp32 model checks a truncated block
        _cache_case("attend_fp32_b3", "attend", 3, 7, 1001, "8/2", 64, 16, "fp32"),
        # one token of one request, with a chat's history
        _logits_case("process_one_b1", "process", 1, 1, 151936, "fp32", 1000, 0, False),
        # a whole block for 64 requests with every kind of processing
        _logits_case("process_block_b64", "process", 64, 16, 151936, "bf16", 4096, 300, True),
        # a greedy check of one block, no processing
        _logits_case("verify_block_b1", "verify", 1, 16, 151936, "fp32", 0, 0, False),
        # sampled verification of 64 blocks with penalties and grammar masks
        _logits_case("verify_block_b64", "verify", 64, 16, 151936, "bf16", 2048, 0, True, 0.8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "process", "verify"])
    if op in ("append", "attend"):
        heads = rng.choice(sorted(HEADS))
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        case = {"op": op, "heads": heads, "dim": rng.choice([64, 128, 128, 256]), "dtype": dtype,
                "page": rng.choice([16, 32, 64, 128]), "window": 0, "sinks": 0}
        batch = _log_int(rng, 1, 64)
        kind = rng.choice(["one", "block", "prompt"])
        new = 1 if kind == "one" else rng.randint(2, 16) if kind == "block" else _log_int(rng, 17, 2048)
        if dtype == "fp32":
            batch, new = min(batch, 8), min(new, 64)
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
    vocab = rng.choice([4096, 5003, 32000, 50257, 151936])
    case = {"op": op, "batch": _log_int(rng, 1, 64), "rows": rng.choice([1, 1, 2, 5, 8, 16, 16]),
            "vocab": vocab, "dtype": rng.choice(["bf16", "fp32"]),
            "history": rng.choice([0, _log_int(rng, 1, 16000)]), "bias": rng.choice([0, 0, _log_int(rng, 1, 300)]),
            "mask": rng.random() < 0.5, "temperature": 0.0}
    if case["dtype"] == "fp32":
        case["batch"] = min(case["batch"], 32)
    if op == "process" and not (case["history"] or case["bias"] or case["mask"]):
        case["history"] = 100
    if op == "verify":
        case["temperature"] = rng.choice([0.0, 0.3, 0.8, 1.0, 1.5])
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


def _hist_lens(case):
    return _spread(case["batch"], case["history"] // 2, case["history"])


def work(case):
    if case["op"] in ("append", "attend"):
        hq, hk = HEADS[case["heads"]]
        size = 2 if case["dtype"] == "bf16" else 4
        d = case["dim"]
        new, total = _lens(case)
        if case["op"] == "append":
            return {"bytes": 4 * sum(new) * hk * d * size, "flops": 0}
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
        return {"bytes": 2 * keys * hk * d * size + 2 * sum(new) * hq * d * size + 4 * sum(new) * hq,
                "flops": 4 * pairs * hq * d}
    rows = case["batch"] * case["rows"]
    size = 2 if case["dtype"] == "bf16" else 4
    v = case["vocab"]
    read = rows * v * size + (rows * ((v + 31) // 32) * 4 if case["mask"] else 0)
    read += sum(_hist_lens(case)) * 4 + case["batch"] * case["bias"] * 8
    if case["op"] == "process":
        return {"bytes": read + rows * v * size, "flops": rows * v}
    if case["temperature"]:
        return {"bytes": read + case["batch"] * v * 4, "flops": 4 * rows * v}
    return {"bytes": read, "flops": rows * v}


# ------------------------------------------------------------------ inputs
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cache_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq, hk = HEADS[case["heads"]]
    d, ps, dt = case["dim"], case["page"], TYPES[case["dtype"]]
    new, total = _lens(case)
    tokens = sum(new)
    pages = [-(-t // ps) for t in total]
    num, width = sum(pages) + 3, max(pages)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    def cache():
        # page by page a cache fills with what its requests wrote; values as a projection gives them
        return torch.empty((num, hk, ps, d), dtype=dt, device="cuda").normal_(generator=g)

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


def _logits_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    b, t, v = case["batch"], case["rows"], case["vocab"]

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    def ids(*shape):  # a few ids are frequent and most are rare, as in text
        return (uniform(*shape) ** 3 * v).long().clamp_(max=v - 1).to(torch.int32)

    logits = torch.randn((b, t, v), generator=g, device="cuda").mul_(2.5)
    # the proposals: the target would mostly have said the same
    draft = ids(b, max(t - 1, 0))
    if t > 1:
        agree = torch.where(uniform(b, t - 1) < 0.85, 14.0, 6.0)
        logits[:, :-1].scatter_add_(2, draft.long()[..., None], agree[..., None])
    state = {"case": case, "logits": logits.to(TYPES[case["dtype"]]), "draft": draft}
    if case["history"]:
        n = _hist_lens(case)
        state.update(history=ids(b, case["history"]), history_len=_ints(n),
                     prompt_len=_ints([x * 2 // 3 for x in n]),
                     repetition=1.0 + 0.3 * uniform(b), frequency=0.2 * uniform(b), presence=0.5 * uniform(b))
    if case["bias"]:
        # distinct ids in each list
        state.update(bias_ids=torch.stack([torch.randperm(v, generator=g, device="cuda")[:case["bias"]]
                                           for _ in range(b)]).to(torch.int32),
                     bias_values=4 * uniform(b, case["bias"]) - 2)
    if case["mask"]:
        # every other request has a grammar that allows about half of the ids, the others allow all
        words = torch.randint(-2 ** 31, 2 ** 31, (b, t, (v + 31) // 32), generator=g, device="cuda")
        words[1::2] = -1
        if t > 1:  # the drafter knew the grammar
            at = (draft.long() // 32)[..., None]
            have = words[:, :-1].gather(2, at) & 0xFFFFFFFF
            have = have | (1 << (draft.long() % 32))[..., None]
            words[:, :-1].scatter_(2, at, torch.where(have >= 2 ** 31, have - 2 ** 32, have))
        state["mask"] = words.to(torch.int32)
    if case["op"] == "verify" and case["temperature"]:
        state.update(temperature=torch.full((b,), case["temperature"], device="cuda"),
                     accept_u=uniform(b, max(t - 1, 0)),
                     noise=torch.empty((b, v), device="cuda").exponential_(generator=g).clamp_(min=1e-30))
    return state


def prepare(case, seed):
    state = _cache_inputs(case, seed) if case["op"] in ("append", "attend") else _logits_inputs(case, seed)
    if own:
        from gru_corrected_draft_amd import verify
        if case["op"] in ("append", "attend"):
            hq, hk = HEADS[case["heads"]]
            state["attention"] = verify.PagedAttention(hq, hk, case["dim"], case["page"], TYPES[case["dtype"]],
                                                       max_requests=case["batch"])
        else:
            state["verifier"] = verify.DraftVerifier(case["vocab"], TYPES[case["dtype"]],
                                                     max_requests=case["batch"], max_rows=case["rows"])
    return state


# ------------------------------------------------------------------ plain forms
def _token_owner(s):
    """Request and cache position of each new token."""
    start, kv = s["q_start"].long(), s["kv_len"].long()
    tokens = (s["k"] if "k" in s else s["q"]).shape[0]
    at = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(start[1:], at, right=True)
    return b, kv[b] - (start[b + 1] - at)


def _plain_append(s):
    ps = s["case"]["page"]
    b, pos = _token_owner(s)
    page = s["page_table"].long()[b, pos // ps]
    s["k_cache"][page, :, pos % ps] = s["k"]
    s["v_cache"][page, :, pos % ps] = s["v"]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


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
    page = s["page_table"].long().gather(1, safe // ps)
    page = page.clamp(min=0)
    k = s["k_cache"][page, :, safe % ps].float()  # [batch, keys, hk, d]
    v = s["v_cache"][page, :, safe % ps].float()
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


def _plain_processed(s):
    """The processed logits in 32 bits."""
    case = s["case"]
    b, t, v = case["batch"], case["rows"], case["vocab"]
    x = s["logits"].float()
    if case["history"]:
        at = torch.arange(case["history"], device="cuda")
        ids = s["history"].long()
        said = ((at >= s["prompt_len"][:, None]) & (at < s["history_len"][:, None])).float()
        asked = (at < s["prompt_len"].minimum(s["history_len"])[:, None]).float()
        count = torch.zeros((b, v), device="cuda").scatter_add_(1, ids, said)
        prompt = torch.zeros((b, v), device="cuda").scatter_add_(1, ids, asked)
        count = count[:, None].repeat(1, t, 1)
        if t > 1:  # a row has seen the proposals before it
            count[:, 1:] += torch.zeros((b, t - 1, v), device="cuda").scatter_(
                2, s["draft"].long()[..., None], 1.0).cumsum_(1)
        seen = (count > 0) | (prompt[:, None] > 0)
        r = s["repetition"][:, None, None]
        x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
        x = x - s["frequency"][:, None, None] * count
        x = x - s["presence"][:, None, None] * (count > 0)
    if case["bias"]:
        x = x.scatter_add(2, s["bias_ids"].long()[:, None].expand(b, t, -1),
                          s["bias_values"][:, None].expand(b, t, -1))
    if case["mask"]:
        bit = torch.arange(32, device="cuda", dtype=torch.int32)
        allowed = ((s["mask"][..., None] >> bit) & 1).view(b, t, -1)[..., :v].bool()
        x = x.masked_fill(~allowed, -math.inf)
    return x


def _plain_verify(s):
    case = s["case"]
    b, t = case["batch"], case["rows"]
    x = _plain_processed(s)
    draft = s["draft"].long()
    warm = case["temperature"] > 0
    temp = case["temperature"] if warm else 1.0
    top = x.amax(-1, keepdim=True)
    logp = (x - top) / temp
    logp = logp - logp.exp().sum(-1, keepdim=True).log()
    score = x - temp * s["noise"].log()[:, None] if warm else x
    if t > 1:
        if warm:
            stands = s["accept_u"] < logp[:, :-1].gather(2, draft[..., None]).squeeze(-1).exp()
            score[:, :-1].scatter_(2, draft[..., None], -math.inf)
        else:
            stands = x[:, :-1].argmax(-1) == draft
        accepted = stands.long().cumprod(1).sum(1)
    else:
        accepted = torch.zeros(b, dtype=torch.long, device="cuda")
    chosen = score[torch.arange(b, device="cuda"), accepted].argmax(-1)
    step = torch.arange(t, device="cuda")
    tokens = torch.cat([draft, draft.new_zeros(b, 1)], 1)
    tokens = torch.where(step == accepted[:, None], chosen[:, None], tokens)
    past = step > accepted[:, None]
    said = logp.gather(2, tokens[..., None]).squeeze(-1)
    return {"tokens": tokens.masked_fill(past, -1).int(), "accepted": accepted.int(),
            "logprob": said.masked_fill(past, 0.0)}


def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "append":
            return _plain_append(s)
        if op == "attend":
            return _plain_attend(s)
        if op == "process":
            return _plain_processed(s).to(s["logits"].dtype)
        return _plain_verify(s)
    case = s["case"]
    if op == "append":
        s["attention"].append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"],
                              s["q_start"], max_new=s["max_new"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "attend":
        out, lse = s["attention"].run(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"],
                                      s["q_start"], max_new=s["max_new"], max_kv=s["max_kv"],
                                      window=case["window"], sinks=case["sinks"], return_lse=True)
        return {"out": out, "lse": lse}
    rules = {n: s.get(n) for n in ("history", "history_len", "prompt_len", "repetition", "frequency",
                                   "presence", "bias_ids", "bias_values", "mask")}
    if op == "process":
        return s["verifier"].process(s["logits"], draft=s["draft"], **rules)
    tokens, accepted, logprob = s["verifier"].run(s["logits"], s["draft"], temperature=s.get("temperature"),
                                                  accept_u=s.get("accept_u"), noise=s.get("noise"),
                                                  return_logprob=True, **rules)
    return {"tokens": tokens, "accepted": accepted, "logprob": logprob}


# ------------------------------------------------------------------ 64 bits, request by request
def _exact_append(s):
    ps = s["case"]["page"]
    kv, start = s["kv_len"].tolist(), s["q_start"].tolist()
    table = s["page_table"].tolist()
    k, v = s["k_cache"].clone(), s["v_cache"].clone()
    for b, n in enumerate(kv):
        fresh = start[b + 1] - start[b]
        for i in range(fresh):
            pos = n - fresh + i
            page, row = table[b][pos // ps], pos % ps
            k[page, :, row] = s["k"][start[b] + i]
            v[page, :, row] = s["v"][start[b] + i]
    return {"k_cache": k.double(), "v_cache": v.double()}


def _exact_attend(s):
    case = s["case"]
    hq, hk = HEADS[case["heads"]]
    w = case["window"]
    start, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    outs, lses = [], []
    for b, n in enumerate(lens):
        pages = s["page_table"][b, :-(-n // case["page"])].long()
        keys = s["k_cache"][pages].transpose(1, 2).reshape(-1, hk, case["dim"])[:n]
        values = s["v_cache"][pages].transpose(1, 2).reshape(-1, hk, case["dim"])[:n]
        q = s["q"][start[b]:start[b + 1]].double()
        place = torch.arange(n, device="cuda")
        mine = torch.arange(n - q.shape[0], n, device="cuda")[:, None]
        hidden = place > mine
        if w:
            hidden |= (mine - place >= w) & (place >= case["sinks"])
        out, lse = torch.empty_like(q), q.new_empty(q.shape[:2])
        for h in range(hq):
            kh, vh = keys[:, h * hk // hq].double(), values[:, h * hk // hq].double()
            a = (torch.mm(q[:, h], kh.t().contiguous()) / case["dim"] ** 0.5).masked_fill(hidden, -math.inf)
            lse[:, h] = torch.logsumexp(a, 1)
            out[:, h] = torch.mm(torch.softmax(a, 1), vh)
        outs.append(out)
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_rows(s, b):
    """The processed rows of request b in 64 bits."""
    case = s["case"]
    x = s["logits"][b].double()
    if case["history"]:
        n, m = int(s["history_len"][b]), int(s["prompt_len"][b])
        h = s["history"][b].long()
        asked = torch.bincount(h[:min(m, n)], minlength=case["vocab"]) > 0
        said = torch.bincount(h[m:n], minlength=case["vocab"])
        r, f, p = (float(s[i][b]) for i in ("repetition", "frequency", "presence"))
        rows = []
        for t in range(case["rows"]):
            if t:
                said[int(s["draft"][b, t - 1])] += 1
            y = x[t]
            y = torch.where(asked | (said > 0), torch.where(y > 0, y / r, y * r), y)
            rows.append(y - f * said - p * (said > 0))
        x = torch.stack(rows)
    if case["bias"]:
        x = x.index_add(1, s["bias_ids"][b].long(), s["bias_values"][b].double().expand(case["rows"], -1))
    if case["mask"]:
        v = torch.arange(case["vocab"], device="cuda")
        x = torch.where((s["mask"][b].long()[:, v // 32] >> (v % 32)) & 1 == 1, x, -math.inf)
    return x


def _exact_verify(s):
    case = s["case"]
    temp = case["temperature"]
    tokens = torch.full((case["batch"], case["rows"]), -1, dtype=torch.int32)
    logprob = torch.zeros((case["batch"], case["rows"]), dtype=torch.float64)
    accepted = torch.zeros(case["batch"], dtype=torch.int32)
    draft = s["draft"].tolist()
    # inputs are 32-bit numbers, the temperature among them
    temp = float(torch.tensor(temp, dtype=torch.float32)) if temp else 0.0
    for b in range(case["batch"]):
        x = _exact_rows(s, b)
        logp = torch.log_softmax(x / (temp or 1.0), 1)
        for t in range(case["rows"]):
            score = x[t] - temp * s["noise"][b].double().log() if temp else x[t]
            if t < case["rows"] - 1:
                at = draft[b][t]
                if (float(s["accept_u"][b, t]) < float(logp[t, at].exp())) if temp else int(x[t].argmax()) == at:
                    tokens[b, t], logprob[b, t] = at, float(logp[t, at])
                    continue
                if temp:
                    score[at] = -math.inf
            accepted[b], tokens[b, t] = t, int(score.argmax())
            logprob[b, t] = float(logp[t, int(tokens[b, t])])
            break
    return {"tokens": tokens, "accepted": accepted, "logprob": logprob}


def exact(case, seed):
    if case["op"] in ("append", "attend"):
        s = _cache_inputs(case, seed)
        return _exact_append(s) if case["op"] == "append" else _exact_attend(s)
    s = _logits_inputs(case, seed)
    if case["op"] == "process":
        return torch.stack([_exact_rows(s, b) for b in range(case["batch"])])
    return _exact_verify(s)
