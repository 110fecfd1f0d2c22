"""The example's decoding step: hidden states to tokens through the 8-bit head and the filtered sampler."""
import os
import subprocess
import sys

import pytest
import torch

import vocab_wide_logit_gb300 as pkg

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def test_step():
    import next_token
    dev = torch.device("cuda", 0)
    rows, vocab, hidden = 40, 5000, 256
    head, weight, gain = next_token.build_head(vocab, hidden, dev)
    params = next_token.settings(rows, dev)
    g = torch.Generator(device=dev).manual_seed(2)
    h = torch.randn((rows, hidden), generator=g, device=dev).to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    tokens, logprobs = next_token.step(head, h, params, torch.rand((rows,), generator=g, device=dev), status)
    assert int(status.item()) == 0
    logits = head.logits(h).double()
    assert bool(((tokens >= 0) & (tokens < vocab)).all())
    assert torch.equal(tokens[0::5].long(), logits[0::5].float().argmax(1))  # greedy requests
    rank = (logits > logits.gather(1, tokens.long()[:, None])).sum(1)
    assert bool((rank[1::5] < 50).all())  # top-k 50
    want = torch.log_softmax(logits, 1).gather(1, tokens.long()[:, None])[:, 0]
    assert float((logprobs.double() - want).abs().max()) <= 1e-4
    # Close to the unquantised head: the logits' spread is about 3; each operand is off by up to half of 1/127 of its
    # row's largest value, about 4 times its rms, so by 4 / 127 / sqrt(12) of its rms: 0.013 times the spread for both.
    y = h.double()
    y = y / torch.sqrt((y * y).mean(1, keepdim=True) + 1e-6) * gain.double()
    real = y @ weight.double().t()
    assert float((logits - real).square().mean().sqrt() / real.square().mean().sqrt()) <= 0.03


def test_runs_as_a_program():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "next_token.py"), "--rows", "7", "--vocab", "3001",
                        "--hidden", "128", "--steps", "2"], capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stderr
    assert r.stdout.count("step ") == 2
