"""Answers to a batch of prompts, each a list of small whole numbers: tokenizer, block table, cached keys and values and the
attention over them, token sets, grammar masks, shaped logits and drawn tokens together, as a serving program runs them.

    python examples/serve_step.py

The model is a stand-in (random logits by last token, row and step, and one layer of attention with random weights); all the rest
is what a server does around one.  Nothing waits for the device inside the loop but the check whether every answer has ended.
"""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import exact_byte_level_amd as tt  # noqa: E402


def number_list():
    """Automaton of '[', whole numbers of up to three digits separated by ', ', ']'."""
    nxt = np.full((7, 256), -1)
    digits = np.arange(48, 58)
    nxt[0, ord("[")] = 1
    nxt[1, digits], nxt[2, digits], nxt[3, digits] = 2, 3, 4
    nxt[2:5, ord(",")] = 5
    nxt[5, ord(" ")] = 1
    nxt[2:5, ord("]")] = 6
    return nxt, np.arange(7) == 6


def answer(prompts, steps=48, seed=0):
    """The answers' bytes to `prompts` (texts as bytes)."""
    tt.load(np.load(os.path.join(ROOT, "data", "vocab_c1.npy")))
    tokens = tt.TokenStrings.of_tokenizer()
    end = tokens.n_tokens            # the model's vocabulary: the tokenizer's, then the end token
    vocab, rows = end + 1, len(prompts)
    nxt, accept = number_list()
    grammar = tt.Grammar(nxt, accept, end_id=end)
    allowed = tt.grammar_bits(grammar, tokens, vocab=vocab)  # of every state, once

    # prompts -> ids, sets of their tokens, blocks of the cache
    bounds = torch.tensor(np.cumsum([0] + [len(p) for p in prompts]), device="cuda")
    text = torch.from_numpy(np.frombuffer(b"".join(prompts), np.uint8).copy()).cuda()
    ids, offsets = tt.encode_batch(text, bounds)
    width = -(-(int(offsets.diff().max()) + steps) // 16)    # room for the longest prompt and its answer
    offsets = offsets.cuda()
    seen = tt.token_bits(ids, vocab, offsets=offsets)
    cache = tt.BlockTable(rows, width=width, blocks=width * rows, block_size=16)
    slots, positions, row_of = cache.plan(offsets)           # where the model puts the prompts' keys and values

    g = torch.Generator("cuda").manual_seed(seed)
    model = torch.randn(vocab, vocab, device="cuda", generator=g).bfloat16()
    heads, kv, dim = 4, 2, 64
    embed, to_q, to_k, to_v, to_logits = (torch.randn(*shape, device="cuda", generator=g).mul_(shape[0]**-0.5).bfloat16() for shape in (
        (vocab, dim), (dim, heads * dim), (dim, kv * dim), (dim, kv * dim), (heads * dim, vocab)))
    layer = tt.KeyValueCache(cache, kv, dim)

    def write(ids, slots):
        x = embed[ids.long()]
        layer.write((x @ to_k).view(-1, kv, dim), (x @ to_v).view(-1, kv, dim), slots)

    write(ids, slots)
    made = torch.zeros(rows, steps, dtype=torch.int32, device="cuda")
    n_made = torch.zeros(rows, dtype=torch.int32, device="cuda")
    states = torch.zeros(rows, dtype=torch.int32, device="cuda")
    live = torch.ones(rows, dtype=torch.bool, device="cuda")
    # the prompts' last tokens; an empty one begins after an end token
    last = torch.cat([ids, ids.new_full((1,), end)])[torch.where(offsets[1:] > offsets[:-1], offsets[1:] - 1, len(ids))].long()
    fixed = {k: torch.full((rows,), v, device="cuda") for k, v in
             dict(repetition=1.2, frequency=0.3, presence=0.1, temperature=0.8, top_p=0.95, min_p=0.02).items()}
    shaping = {k: fixed[k] for k in ("repetition", "frequency", "presence", "temperature")}
    # closing gets likelier than random logits make it
    closing = dict(bias_offsets=torch.arange(rows + 1, device="cuda"), bias_values=torch.full((rows,), 1.5, device="cuda"),
                   bias_ids=torch.full((rows,), ord("]"), dtype=torch.int32, device="cuda"))
    slot, count = (torch.empty(n, dtype=torch.int64, device="cuda") for n in (rows, 1))
    for step in range(steps):
        logits = model[(last + 97 * torch.arange(rows, device="cuda") + step) % vocab]
        seen_before = layer.attend((embed[last] @ to_q).view(rows, heads, dim))  # the last token over all that its row has cached
        logits = logits + seen_before.view(rows, -1) @ to_logits
        out = tt.shape_logits(logits, seen=seen, generated=made, n_generated=n_made, allowed=allowed, allowed_rows=states,
                              **shaping, **closing)
        chosen = tt.sample_tokens(out, torch.rand(rows, device="cuda", generator=g), top_p=fixed["top_p"], min_p=fixed["min_p"])
        ended = live & (chosen == end)
        live &= ~ended
        cache.release_into(ended, count)
        tt.grammar_advance_into(grammar, tokens, states, torch.where(live, chosen, -1))
        made.scatter_(1, n_made[:, None].clamp(max=steps - 1).long(), torch.where(live, chosen, made[:, -1])[:, None])
        n_made += live.int()
        cache.plan_into(slot, count)                         # a slot for each live answer's next token, -1 for the others
        last = torch.where(live, chosen.long(), last)
        write(last, slot)
        if not bool(live.any()):
            break
    strings, off = tokens.strings.cpu().numpy().tobytes(), tokens.offsets.tolist()
    made, n_made = made.tolist(), n_made.tolist()
    return [b"".join(strings[off[t]:off[t + 1]] for t in made[r][:n_made[r]]) for r in range(rows)], ~live


def main():
    prompts = [b"Name three primes.", b"def f(n):\n    return", b"1 2 3", b"The years of the eclipses were"]
    answers, ended = answer(prompts)
    for p, a, e in zip(prompts, answers, ended.tolist()):
        print("%r -> %s%s" % (p.decode(), a.decode(), "" if e else " ..."))


if __name__ == "__main__":
    main()
