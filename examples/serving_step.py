"""One request served token by token with speculative verification, around the
weight stream: block tables, the norms, rotation and 8-bit cache write of an
attention layer, attention over the cache, the layer's NVFP4 projections, the FP8
output layer and the verification of drafted tokens. Random weights, and a drafter
that is the model without its attention; what it shows is how the calls fit
together.

    python examples/serving_step.py [--steps 8] [--drafts 3]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_streaming_gb300 as bws  # noqa: E402
import synth  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM, VOCAB, BLOCK = 1024, 8, 2, 128, 32000, 16


def int32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


class Model:
    """One attention layer and the output layer, weights quantized by this library."""

    def __init__(self, dev, seed=0):
        def nvfp4(shape, i):
            return bws.nvfp4_quantize(synth.weight_fp32(shape, seed=seed, index=i, device=dev))

        self.qkv = nvfp4(((Q_HEADS + 2 * KV_HEADS) * DIM, HIDDEN), 0)
        self.out = nvfp4((HIDDEN, Q_HEADS * DIM), 1)
        self.head = bws.fp8_rowwise_quantize(synth.weight_fp32((VOCAB, HIDDEN), seed=seed, index=2, std=0.1, device=dev))
        self.embed = synth.weight_fp32((VOCAB, HIDDEN), seed=seed, index=3, std=1.0, device=dev).to(torch.bfloat16)
        self.q_norm, self.k_norm = torch.ones(DIM, device=dev), torch.ones(DIM, device=dev)
        self.inv_freq = (1e4 ** (-torch.arange(0, DIM, 2, device=dev, dtype=torch.float64) / DIM)).float()
        self.cache = bws.KvCache.empty(64, KV_HEADS, DIM, BLOCK, dev)
        self.ws = bws.Workspace(dev)

    def probabilities(self, tokens, table, plan, rows):
        """Next-token probabilities after each of the rows' tokens, which enter the cache."""
        x = self.embed[tokens.long()]
        y = bws.nvfp4_gemv(*self.qkv, x, ws=self.ws).view(-1, Q_HEADS + 2 * KV_HEADS, DIM)
        q = bws.qk_norm_rope_append(y[:, :Q_HEADS], y[:, Q_HEADS:Q_HEADS + KV_HEADS], y[:, Q_HEADS + KV_HEADS:],
                                    plan.positions, plan.slots, self.cache, self.inv_freq, self.q_norm, self.k_norm)
        a = bws.kv_attention(q, self.cache, table, plan.row_start, plan.kv_lens, rows, ws=self.ws)
        x = x + bws.nvfp4_gemv(*self.out, a.view(-1, Q_HEADS * DIM), ws=self.ws)
        return torch.softmax(bws.fp8_lmhead_gemv(*self.head, x, ws=self.ws), -1)

    def draft(self, token, n):
        """n tokens drawn one after the other from the output layer on the embedding, and their probabilities."""
        tokens, probs = [], []
        for _ in range(n):
            probs.append(torch.softmax(bws.fp8_lmhead_gemv(*self.head, self.embed[token][None], ws=self.ws), -1))
            token = torch.multinomial(probs[-1][0], 1).item()
            tokens.append(token)
        return tokens, probs


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=3)
    a = ap.parse_args()
    dev, rows = torch.device("cuda:0"), a.drafts + 1
    assert 1 <= rows <= 8, "a verify pass takes up to eight tokens"
    torch.manual_seed(0)
    model = Model(dev)
    table = torch.full((1, 64), -1, dtype=torch.int32, device=dev)
    free, n_free = int32(list(range(64)), dev), int32([64], dev)
    seq, text = 0, [1]                        # tokens in the cache; the text, whose last token is not yet in it
    for _ in range(a.steps):
        drafts, probs = model.draft(text[-1], a.drafts)
        tokens = int32([text[-1]] + drafts, dev)
        plan = bws.kv_plan(int32([seq], dev), int32([rows], dev), BLOCK, table, free, n_free, rows)
        target = model.probabilities(tokens, table, plan, rows)
        draft = torch.cat(probs + [torch.zeros_like(target[:1])])
        # row i drafted the token of row i + 1; the last row drafted none
        out, n = bws.draft_verify(target, torch.roll(tokens, -1), plan.row_start, torch.rand(rows, device=dev),
                                  torch.rand(1, device=dev), rows, draft=draft)
        new = out[0, :n.item()].tolist()
        text += new
        # the tokens that stand are in the cache already; the drawn one enters with the next step. Blocks the
        # plan took stay with the request: its table row keeps them, and n_free counts them as taken.
        seq += len(new)
        held = -(-(seq - len(new) + rows) // BLOCK)
        if held > -(-seq // BLOCK):           # a whole block of refused drafts goes back
            plan.n_free.add_(held - -(-seq // BLOCK))
        n_free = plan.n_free
    print(f"{a.steps} steps of {rows} tokens: {len(text) - 1} tokens; status {bws.status_word(model.ws)}; "
          f"free blocks {n_free.item()}; text {text}")
    return text


if __name__ == "__main__":
    main()
