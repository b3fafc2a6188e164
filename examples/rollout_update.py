"""Sampling, scoring and two updates of an LM head: how the library's calls go together.

A toy policy is an LM head over fixed hidden states. One round
  1. lays its weight out in 8 bits and samples a token for every hidden state through the
     8-bit head and the sampler, with the tokens' logprobs (the rollout);
  2. scores those tokens under the reference head;
  3. rewards the tokens of one half of the vocabulary and takes the clipped policy loss
     with its KL term and the logits' gradient, and a step on the weight;
  4. makes pairs of short answers from the same tokens, the better one first, and takes a
     step on the preference loss.

    python examples/rollout_update.py        (needs a GB300)
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from decode_step_token_gb300 import Sampler  # noqa: E402


class Head:
    """An LM head [vocab, width] in bf16, and its 8-bit form for rollouts."""

    def __init__(self, sampler: Sampler, weight: torch.Tensor):
        self.sampler, self.weight = sampler, weight
        vocab, width = weight.shape
        self.values = torch.empty((vocab, width), dtype=torch.float8_e4m3fn, device=weight.device)
        self.scales = torch.empty((-(-vocab // 128), -(-width // 128)), device=weight.device)
        self.lay_out()

    def lay_out(self) -> None:
        self.sampler.quantize_blocks(src=self.weight, block_rows=128, out_values=self.values, out_scales=self.scales)

    def eight(self, hidden: torch.Tensor) -> dict:
        """The operands of the 8-bit head for these hidden states."""
        values = torch.empty(hidden.shape, dtype=torch.float8_e4m3fn, device=hidden.device)
        scales = torch.empty((hidden.shape[0], self.scales.shape[1]), device=hidden.device)
        self.sampler.quantize_blocks(src=hidden, block_rows=1, out_values=values, out_scales=scales)
        return dict(hidden=values, hidden_scale=scales, weight=self.values, weight_scale=self.scales)


def run(rows: int = 64, vocab: int = 4096, width: int = 256, rounds: int = 4, seed: int = 0) -> list:
    """The mean reward of each round's rollout."""
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(seed)
    sampler = Sampler(max_rows=rows, max_vocab=vocab)
    hidden = torch.randn((rows, width), generator=gen, device=dev).to(torch.bfloat16)
    weight = (torch.randn((vocab, width), generator=gen, device=dev) / width ** 0.5).to(torch.bfloat16)
    policy, reference = Head(sampler, weight.clone()), weight.clone()
    master = policy.weight.float()  # the step is taken in fp32
    temperature = torch.ones(rows, device=dev)
    tokens = torch.empty(rows, dtype=torch.int32, device=dev)
    old, ref = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    loss, entropy = torch.empty(1, device=dev), torch.empty(rows, device=dev)
    logits = torch.empty((rows, vocab), dtype=torch.bfloat16, device=dev)
    grad = torch.empty_like(logits)
    mean_weight = torch.full((rows,), 1.0 / rows, device=dev)
    rewards = []

    def step(rate: float) -> None:
        master.sub_(rate * (grad.float().t() @ hidden.float()))
        policy.weight.copy_(master)

    for r in range(rounds):
        # the rollout: 8-bit head, sampled token, its logprob
        args = sampler.make_args(logits=logits, temperature=temperature, out_tokens=tokens, philox_offset=r)
        sampler.lm_head_scaled_sample_args(args, out_token_logprob=old, **policy.eight(hidden))
        # the same tokens under the reference
        torch.matmul(hidden, reference.t(), out=logits)
        sampler.score(logits=logits, tokens=tokens, temperature=temperature, out_logprob=ref, out_entropy=entropy)
        # tokens of the lower half of the vocabulary are wanted
        reward = (tokens < vocab // 2).float()
        rewards.append(reward.mean().item())
        torch.matmul(hidden, policy.weight.t(), out=logits)
        sampler.policy_loss(logits=logits, tokens=tokens, temperature=temperature, weight=mean_weight, old_logprob=old,
                            advantage=2.0 * reward - 1.0, ref_logprob=ref, kl_coef=0.01, clip_low=0.2, clip_high=0.3,
                            out_loss=loss, out_grad=grad)
        step(4.0)
        # answers of four tokens, the one with more wanted tokens first in its pair
        answer = torch.arange(rows, device=dev).view(-1, 2, 4)
        worse_first = reward[answer].sum(2)[:, 0] < reward[answer].sum(2)[:, 1]
        order = torch.where(worse_first[:, None, None], answer.flip(1), answer).reshape(-1)
        ends = torch.arange(0, rows + 1, 4, dtype=torch.int32, device=dev)
        torch.matmul(hidden[order], policy.weight.t(), out=logits)
        sampler.preference_loss(logits=logits, tokens=tokens[order], seq_offsets=ends, ref_logprob=ref[order], beta=0.5,
                                out_loss=loss, out_grad=grad)
        grad.copy_(grad[torch.argsort(order)])
        step(2.0)
        policy.lay_out()
    sampler.close()
    return rewards


if __name__ == "__main__":
    for r, x in enumerate(run()):
        print(f"round {r}: {100 * x:.0f} % of the tokens wanted")
