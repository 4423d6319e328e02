"""64-bit references of the operators of ``domino_verify.h``, in NumPy, one request, row and rule at a
time, with the error bounds that their tests use.  No code of the package is imported."""
import numpy as np

NEG = -np.inf


# ------------------------------------------------------------------ attention
def visible(n_keys, pos, window, sinks):
    """Key positions visible to a token at ``pos``."""
    j = np.arange(n_keys)
    ok = j <= pos
    if window:
        ok &= (j > pos - window) | (j < sinks)
    return ok


def attention(q, keys, values, kv_len, window=0, sinks=0, scale=None):
    """One request: q [new, hq, d], keys and values [kv_len, hk, d] in token order.  Returns out, lse and
    for each (token, head) A = sum_j p_j |v_j| and the largest scale * sum_i |q_i k_ji|."""
    q, keys, values = (np.asarray(x, np.float64) for x in (q, keys, values))
    new, hq, d = q.shape
    hk = keys.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out, lse = np.zeros((new, hq, d)), np.full((new, hq), NEG)
    weight, reach = np.zeros((new, hq, d)), np.zeros((new, hq))
    for t in range(new):
        ok = visible(kv_len, kv_len - new + t, window, sinks)
        if not ok.any():
            continue
        for h in range(hq):
            k, v = keys[ok, h * hk // hq], values[ok, h * hk // hq]
            s = scale * (k @ q[t, h])
            m = s.max()
            p = np.exp(s - m)
            lse[t, h] = m + np.log(p.sum())
            p /= p.sum()
            out[t, h] = p @ v
            weight[t, h] = p @ np.abs(v)
            reach[t, h] = (scale * (np.abs(k) @ np.abs(q[t, h]))).max()
    return out, lse, weight, reach


def attention_bounds(out, weight, reach, kv_len, d, bf16):
    """How far fp32 arithmetic may be from 64 bits.

    A score is a d-term fp32 sum of exact products: off by at most d 2^-24 reach, once more for the scaling
    and the exponential's argument, whose own error is a few 2^-24 of the argument (at most 2 reach).
    Scores off by e change every weight by at most a factor e^(2 e), the sums over the keys add kv_len
    2^-24 each (numerator and denominator) and the exponential a few ulp.  For bf16 each weight is rounded
    (2^-8 at most) and so is the result."""
    u = 2.0 ** -24
    e = u * (d + 8) * reach
    rel = 2 * e + u * (2 * kv_len + 32)
    tol = rel[..., None] * (weight + np.abs(out))
    if bf16:
        tol = tol + 2.0 ** -8 * weight * (1 + rel[..., None]) + 2.0 ** -8 * (np.abs(out) + tol + 2.0 ** -8 * weight)
    # the scale and the statistics themselves are rounded once to fp32
    return tol + 1e-37, e + u * (kv_len + 32) + u * 4 * reach


# ------------------------------------------------------------------ logits
def processed(logits, b, rules, vocab):
    """Rows of request b after the rules, in 64 bits, and an error bound of the fp32 evaluation."""
    x = np.asarray(logits[b], np.float64).copy()
    rows = x.shape[0]
    u = 2.0 ** -23
    tol = np.zeros_like(x)
    r = rules
    draft = r.get("draft")
    n_draft = 0
    if draft is not None and rows > 1:
        n_draft = int(np.clip(r["draft_len"][b] if r.get("draft_len") is not None else rows - 1, 0, rows - 1))
    pen = [r.get(k) for k in ("repetition", "frequency", "presence")]
    if any(p is not None for p in pen):
        rep = 1.0 if pen[0] is None else float(pen[0][b])
        freq = 0.0 if pen[1] is None else float(pen[1][b])
        pres = 0.0 if pen[2] is None else float(pen[2][b])
        prompt, count = np.zeros(vocab, bool), np.zeros(vocab, np.int64)
        if r.get("history") is not None:
            width = r["history"].shape[1]
            n = int(np.clip(width if r.get("history_len") is None else r["history_len"][b], 0, width))
            m = int(np.clip(0 if r.get("prompt_len") is None else r["prompt_len"][b], 0, width))
            for i in range(n):
                v = int(r["history"][b, i])
                if 0 <= v < vocab:
                    if i < m:
                        prompt[v] = True
                    else:
                        count[v] += 1
        for t in range(rows):
            if 0 < t <= n_draft and 0 <= draft[b, t - 1] < vocab:
                count[draft[b, t - 1]] += 1
            seen = prompt | (count > 0)
            y = x[t]
            if pen[0] is not None:
                y = np.where(seen, np.where(y > 0, y / rep, y * rep), y)
            with np.errstate(invalid="ignore"):
                z = y - freq * count - pres * (count > 0)
                tol[t] = u * 4 * (np.abs(y) + np.abs(freq * count) + np.abs(pres))
            x[t] = z
    if r.get("bias_ids") is not None:
        width = r["bias_ids"].shape[1]
        n = int(np.clip(width if r.get("bias_len") is None else r["bias_len"][b], 0, width))
        last = {}
        for i in range(n):
            v = int(r["bias_ids"][b, i])
            if 0 <= v < vocab:
                last[v] = float(r["bias_values"][b, i])
        for v, y in last.items():
            with np.errstate(invalid="ignore"):
                tol[:, v] += u * (np.abs(x[:, v]) + abs(y))
            x[:, v] += y
    if r.get("mask") is not None:
        v = np.arange(vocab)
        words = np.asarray(r["mask"][b]).astype(np.int64) & 0xFFFFFFFF
        x = np.where((words[:, v // 32] >> (v % 32)) & 1 == 1, x, NEG)
    return x, np.where(np.isfinite(tol), tol, 0.0), n_draft


def verify(logits, rules, vocab, temperature=None, accept_u=None, noise=None):
    """Tokens, accepted counts, log-probabilities and the smallest margin of a decision: how near a test
    of a proposal, or the choice of a token, came to going the other way (in units of the logits)."""
    B, rows = logits.shape[:2]
    tokens, accepted = np.full((B, rows), -1, np.int64), np.zeros(B, np.int64)
    logprob, margin = np.zeros((B, rows)), np.inf
    big = float(np.finfo(np.float32).max)
    for b in range(B):
        x, tol, n = processed(logits, b, rules, vocab)
        x = np.where(np.isnan(x), NEG, np.minimum(x, big))
        T = 0.0 if temperature is None else float(temperature[b])
        T = min(max(T, 1e-30), 1e30) if T > 0 else 0.0
        for t in range(n + 1):
            row = x[t]
            m = row.max()
            some = m > NEG
            if some:
                with np.errstate(over="ignore"):
                    z = (row - m) / (T or 1.0)
                lp = z - np.log(np.exp(z).sum())
            score = row.copy()
            if T:
                score = np.where(row > NEG, row - T * np.log(np.asarray(noise[b], np.float64)), NEG)
            if t < n:
                d = int(rules["draft"][b, t])
                if 0 <= d < vocab and row[d] > NEG:
                    others = score.copy()
                    others[d] = NEG
                    if not (others > NEG).any():
                        stands = True
                    elif T:
                        stands = accept_u[b, t] < np.exp(lp[d])
                        margin = min(margin, abs(float(accept_u[b, t]) - np.exp(lp[d])))
                    else:
                        stands = int(np.argmax(row)) == d
                    if stands:
                        tokens[b, t], logprob[b, t] = d, lp[d]
                        accepted[b] += 1
                        continue
                    if T:
                        score[d] = NEG
            if not some or not (score > NEG).any():
                logprob[b, t] = NEG
            else:
                tokens[b, t] = int(np.argmax(score))
                logprob[b, t] = lp[tokens[b, t]]
                top = np.sort(score[score > NEG])[-2:]
                if len(top) == 2 and top[1] != top[0]:
                    margin = min(margin, top[1] - top[0])
            break
    return tokens, accepted, logprob, margin
