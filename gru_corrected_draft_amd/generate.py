"""Generation with draft blocks: the rollout proposes, a target model checks the block in one pass.

``python -m gru_corrected_draft_amd.generate`` runs it with random weights.  The loop is what a
server would do with the operators of ``verify``; the target here is a small decoder whose matrix
products are torch's.  A block costs one pass over 16 positions of each request:

1. the drafter proposes 15 tokens after the last verified one;
2. keys and values of the verified token and the proposals are appended to the paged cache, and the
   16 tokens attend to it;
3. the rules apply to the 16 rows of logits, proposals are accepted from the front, and the token
   after the last accepted one is chosen;
4. the lengths advance by what was accepted.  Keys of refused proposals stay in their pages: they lie
   past the new length, where no token sees them, and the next block overwrites them.

Lengths, page tables and texts stay on the GPU; the host only knows bounds for them.  A block may add
16 tokens to a text and often adds few, so the bound runs ahead of the lengths; where it leaves no room
for a block, the longest length is read back once.
"""
from __future__ import annotations

import argparse

import torch

from .rollout import N_PROPOSALS
from .verify import DraftVerifier, PagedAttention

BLOCK = N_PROPOSALS + 1


def _norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Target:
    """A small decoder with random weights: embedding and position, layers of attention and a gated
    product, a head over the vocabulary.  Every second layer sees a window and four sinks."""

    def __init__(self, vocab, hidden, q_heads, kv_heads, head_dim, layers, positions, window=0,
                 dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)

        def weight(rows, cols, scale=1.0):
            return (torch.randn(rows, cols, generator=g) * (scale * cols ** -0.5)).to(device, dtype)

        self.vocab, self.hidden, self.dtype, self.device = vocab, hidden, dtype, device
        self.heads, self.window = (q_heads, kv_heads, head_dim), window
        self.embed = torch.randn(vocab, hidden, generator=g).to(device, dtype)
        self.position = torch.randn(positions, hidden, generator=g).to(device, dtype)
        self.head = weight(vocab, hidden, 4.0)
        self.layers = [{"qkv": weight((q_heads + 2 * kv_heads) * head_dim, hidden),
                        "out": weight(hidden, q_heads * head_dim),
                        "up": weight(4 * hidden, hidden), "down": weight(hidden, 2 * hidden)}
                       for _ in range(layers)]

    def forward(self, tokens, positions, attention, caches, where, bounds):
        """Hidden states of ``tokens`` ([n]) at ``positions``, whose keys and values join the caches
        (one pair a layer).  ``where`` is (page_table, kv_len, q_start), ``bounds`` (max_new, max_kv)."""
        q_heads, kv_heads, dim = self.heads
        x = self.embed[tokens] + self.position[positions]
        for i, (w, (k_cache, v_cache)) in enumerate(zip(self.layers, caches)):
            # q, k and v are views of one product: the operators take any strides
            qkv = (_norm(x) @ w["qkv"].T).view(len(tokens), q_heads + 2 * kv_heads, dim)
            q, k, v = qkv.split([q_heads, kv_heads, kv_heads], 1)
            attention.append(k, v, k_cache, v_cache, *where, *bounds)
            windowed = self.window > 0 and i % 2 == 1
            o = attention.run(q, k_cache, v_cache, *where, *bounds, window=self.window if windowed else 0,
                              sinks=4 if windowed else 0)
            x = x + o.flatten(1) @ w["out"].T
            a, b = (_norm(x) @ w["up"].T).chunk(2, -1)
            x = x + (torch.nn.functional.silu(a) * b) @ w["down"].T
        return _norm(x)


class Generator:
    """Texts of a batch and what the target has cached of them.

    ``rules`` are keyword arguments of ``DraftVerifier.process`` that hold for the whole text:
    repetition, frequency, presence, bias_ids, bias_values, mask ([requests, 1, words], for every row).
    ``temperature`` [requests] samples.
    """

    def __init__(self, target, prompts, max_new, page_size=16, rules=None, temperature=None, seed=0):
        self.target, self.rules, self.temperature = target, rules or {}, temperature
        q_heads, kv_heads, dim = target.heads
        dev, b = target.device, len(prompts)
        self.requests = b
        lens = [len(p) for p in prompts]
        if not lens or min(lens) < 1:
            raise ValueError("a prompt needs a token")
        for p in prompts:  # as an index on the GPU, one would end the process
            ids = torch.as_tensor(p)
            if int(ids.min()) < 0 or int(ids.max()) >= target.vocab:
                raise ValueError(f"a prompt's ids must be in [0, {target.vocab})")
        # a block may write up to 15 refused positions past the text
        self.max_kv = max(lens) + max_new + BLOCK
        if self.max_kv > len(target.position):
            raise ValueError("the target has no positions for texts of this length")
        pages = -(-self.max_kv // page_size)
        self.attention = PagedAttention(q_heads, kv_heads, dim, page_size, target.dtype, max_requests=b)
        self.verifier = DraftVerifier(target.vocab, target.dtype, max_requests=b, max_rows=BLOCK)
        self.caches = [tuple(torch.zeros(b * pages, kv_heads, page_size, dim, dtype=target.dtype, device=dev)
                             for _ in range(2)) for _ in target.layers]
        self.random = torch.Generator(dev).manual_seed(seed)
        order = torch.randperm(b * pages, generator=torch.Generator().manual_seed(seed))
        self.page_table = order.to(dev, torch.int32).view(b, pages)
        self.text = torch.full((b, self.max_kv), -1, dtype=torch.int32, device=dev)
        for i, p in enumerate(prompts):
            self.text[i, :len(p)] = torch.as_tensor(p, dtype=torch.int32)
        self.prompt_len = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.length = self.prompt_len.clone()  # of the text; its last token is not in the cache yet
        self.longest = max(lens)  # what the host knows of it: no text is longer
        self._ahead = False       # whether blocks have run since that was a text's own length

        # the prompts, all but their last tokens, in one ragged pass
        cached = [n - 1 for n in lens]
        if max(cached) > 0:
            start = torch.tensor([0] + cached).cumsum(0).to(dev, torch.int32)
            tokens = torch.cat([self.text[i, :n] for i, n in enumerate(cached)]).long()
            pos = torch.cat([torch.arange(n, device=dev) for n in cached])
            target.forward(tokens, pos, self.attention, self.caches,
                           (self.page_table, self.length - 1, start), (max(cached), max(cached)))

    def logits(self, tokens):
        """Logits of ``tokens`` [requests, n], which stand from each text's last position on."""
        b, n = tokens.shape
        first = self.length - 1
        pos = first.long()[:, None] + torch.arange(n, device=tokens.device)
        start = torch.arange(b + 1, dtype=torch.int32, device=tokens.device) * n
        # an id outside the vocabulary is never accepted, whatever it is looked up as
        ids = tokens.flatten().long().clamp(0, self.target.vocab - 1)
        x = self.target.forward(ids, pos.flatten(), self.attention, self.caches,
                                (self.page_table, first + n, start), (n, min(self.longest - 1 + n, self.max_kv)))
        self.hidden = x.view(b, n, -1)
        return (x @ self.target.head.T).view(b, n, -1)

    def last(self):
        return self.text.gather(1, (self.length - 1).long()[:, None])

    def _rules(self, rows):
        rules = dict(history=self.text, history_len=self.length, prompt_len=self.prompt_len, **self.rules)
        if "mask" in rules:
            rules["mask"] = rules["mask"].expand(-1, rows, -1)
        return rules

    def candidates(self, n):
        """The ``n`` likeliest next tokens under the rules: (log-probabilities, ids).  The text stays."""
        x = self.verifier.process(self.logits(self.last()), **self._rules(1))
        return x[:, 0].float().log_softmax(-1).topk(n)

    def block(self, proposals=None):
        """One pass: checks ``proposals`` [requests, up to 15] (None: none) and extends the texts.
        Returns (tokens [requests, n + 1], -1 after the last new one, accepted [requests])."""
        b, dev = self.requests, self.text.device
        rows = 1 if proposals is None else proposals.shape[1] + 1
        if self.longest + rows > self.max_kv and self._ahead:
            self.longest, self._ahead = int(self.length.max()), False
        if self.longest + rows > self.max_kv:
            raise ValueError("the texts may outgrow max_new")
        tokens = self.last() if proposals is None else torch.cat([self.last(), proposals], 1)
        logits = self.logits(tokens)
        noise = u = None
        if self.temperature is not None:
            noise = torch.empty(b, self.target.vocab, device=dev).exponential_(generator=self.random)
            noise.clamp_(min=1e-30)
            if proposals is not None:
                u = torch.rand(b, proposals.shape[1], device=dev, generator=self.random)
        new, accepted = self.verifier.run(logits, proposals, temperature=self.temperature, accept_u=u,
                                          noise=noise, **self._rules(rows))
        # the new tokens into the text; a column past them is written back as it was
        at = self.length.long()[:, None] + torch.arange(new.shape[1], device=dev)
        self.text.scatter_(1, at, torch.where(new >= 0, new, self.text.gather(1, at)))
        self.length = self.length + (new >= 0).sum(1, dtype=torch.int32)
        self.longest += rows
        self._ahead = True
        return new, accepted


def main(argv=None):
    p = argparse.ArgumentParser(description="Generate with draft blocks, random weights.")
    p.add_argument("--requests", type=int, default=4)
    p.add_argument("--prompt", type=int, default=200, help="tokens of the longest prompt")
    p.add_argument("--blocks", type=int, default=6)
    p.add_argument("--k", type=int, default=256, help="the rollout's candidates (0: the vocabulary)")
    p.add_argument("--temperature", type=float, default=0.0)
    args = p.parse_args(argv)

    from . import synth
    from .rollout import DominoRollout, device_weights
    shape = synth.custom_shape(5003, 256, 128, 128, 128, "bf16", 77, name="generate")
    drafter = DominoRollout(device_weights(synth.make_weights(shape)), max_batch=args.requests, max_k=args.k)
    target = Target(shape.vocab, shape.hidden, 8, 2, 64, 4, args.prompt + BLOCK * (args.blocks + 2), window=64)
    b, dev = args.requests, target.device
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, shape.vocab, (max(1, args.prompt * (i + 1) // b),), generator=g).tolist()
               for i in range(b)]
    rules = dict(repetition=torch.full((b,), 1.1, device=dev), presence=torch.full((b,), 0.2, device=dev))
    temperature = torch.full((b,), args.temperature, device=dev) if args.temperature > 0 else None
    gen = Generator(target, prompts, BLOCK * (args.blocks + 1), rules=rules, temperature=temperature)
    logprob, ids = gen.candidates(3)
    print("likeliest first tokens:", ids.tolist())
    # the drafter's hidden states: the target's at the last token, moved by a vector for each position
    moves = torch.randn(N_PROPOSALS, shape.hidden, generator=g).to(dev, torch.bfloat16)
    step_s = torch.zeros(b, N_PROPOSALS - 1, shape.proj_dim, device=dev)
    for i in range(args.blocks):
        hidden = (gen.hidden[:, -1:] + moves).contiguous()
        proposals, _ = drafter.run(hidden, step_s, gen.last()[:, 0].contiguous(), args.k)
        tokens, accepted = gen.block(proposals)
        print(f"block {i}: accepted {accepted.tolist()}, lengths {gen.length.tolist()}")
    drafter.close()
    return gen


if __name__ == "__main__":
    main()
