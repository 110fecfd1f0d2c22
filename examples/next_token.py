"""One decoding step of a serving program, from hidden states to tokens.

A model's output head in 8 bits (final RMS norm, vocabulary projection) and the sampler behind it: hidden states of a
batch of requests with settings of their own become one token and one log-probability each. With --adapters some requests
have a low-rank adapter on the projection; with --alternatives each token comes with its rank and the most likely ones.
Weights and hidden states are random; a serving program has them from its model.

    python examples/next_token.py [--rows 24] [--vocab 32000] [--hidden 1024] [--steps 4] [--adapters 3] [--alternatives 5]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import vocab_wide_logit_gb300 as ds  # noqa: E402


def build_head(vocab, hidden, device, seed=0):
    """The vocabulary projection [vocab, hidden] quantised a scale per token id, and the norm's gain."""
    g = torch.Generator(device=device).manual_seed(seed)
    weight = torch.randn((vocab, hidden), generator=g, device=device) * (3.0 / hidden ** 0.5)
    gain = 1.0 + 0.1 * torch.randn((hidden,), generator=g, device=device)
    return ds.Int8Head.from_weight(weight, gain=gain), weight, gain


def settings(rows, device):
    """Per-request sampling settings: greedy, top-k, nucleus, min-p and plain requests side by side."""
    kind = torch.arange(rows, device=device) % 5
    temperature = torch.where(kind == 0, 0.0, torch.where(kind == 1, 0.7, 1.0)).float()
    top_k = torch.where(kind == 1, 50, 0).to(torch.int32)
    top_p = torch.where(kind == 2, 0.9, 1.0).float()
    min_p = torch.where(kind == 3, 0.05, 0.0).float()
    return temperature, top_k, top_p, min_p


def build_adapters(count, rank, vocab, hidden, device, seed=3):
    """A stack of low-rank adapters of the projection, each a hundredth of it in size."""
    g = torch.Generator(device=device).manual_seed(seed)
    a = (torch.randn((count, rank, hidden), generator=g, device=device) * hidden ** -0.5).to(torch.bfloat16)
    b = torch.randn((count, vocab, rank), generator=g, device=device).to(torch.bfloat16)
    return ds.Adapters(a, b, torch.full((count,), 0.03 * rank ** -0.5, device=device))


def step(head, hidden, params, u, status=None, adapters=None, adapter_ids=None):
    """Tokens int32 [rows] and log-probabilities float32 [rows] of one decoding step."""
    temperature, top_k, top_p, min_p = params
    return head.sample(hidden, temperature, u, top_k=top_k, top_p=top_p, min_p=min_p, d_status=status, adapters=adapters,
                       adapter_ids=adapter_ids)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=24)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--adapters", type=int, default=0)
    ap.add_argument("--alternatives", type=int, default=0)
    a = ap.parse_args()
    device = torch.device("cuda")
    head, _, _ = build_head(a.vocab, a.hidden, device)
    params = settings(a.rows, device)
    adapters = ids = None
    if a.adapters:
        adapters = build_adapters(a.adapters, 16, a.vocab, a.hidden, device)
        ids = (torch.arange(a.rows, device=device) % (a.adapters + 1) - 1).to(torch.int32)  # -1: none
    status = torch.zeros(1, dtype=torch.int32, device=device)
    g = torch.Generator(device=device).manual_seed(1)
    for i in range(a.steps):
        hidden = torch.randn((a.rows, a.hidden), generator=g, device=device).to(torch.bfloat16)
        u = torch.rand((a.rows,), generator=g, device=device)
        tokens, logprobs = step(head, hidden, params, u, status, adapters, ids)
        print("step %d: tokens %s ... logprobs %s ..." % (i, tokens[:6].tolist(),
                                                          ["%.2f" % v for v in logprobs[:6].tolist()]))
        if a.alternatives:
            r = head.score(hidden, tokens, top=a.alternatives, d_status=status, adapters=adapters, adapter_ids=ids)
            print("  request 0: rank %d, entropy %.2f, alternatives %s" % (int(r.ranks[0]), float(r.entropy[0]),
                  ["%d: %.2f" % (t, v) for t, v in zip(r.top_ids[0].tolist(), r.top_logprobs[0].tolist())]))
    if int(status.item()):
        raise SystemExit("the kernels reported input errors: status %d" % int(status.item()))


if __name__ == "__main__":
    main()
