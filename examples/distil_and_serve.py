"""A student LM head learns from a teacher's most likely tokens and is served in 4 bits.

A toy teacher and a toy student are LM heads over the same hidden states. One round
  1. takes the teacher's most likely tokens for every hidden state, their logprobs and the
     logprob of all other tokens together: all that is kept of its logits;
  2. takes the student's divergence from those lists, with a share of the loss of the
     teacher's first token, and the logits' gradient, and a step on the student's weight.
Then the student's weight is laid out in 4 bits, and tokens are generated with it: the hidden
states to 4 bits, the 4-bit head chained to the sampler, and the chosen tokens' rows of the
same weight, read back from the 4 bits, as the next hidden states (a tied embedding).

    python examples/distil_and_serve.py        (needs a GB300)
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from decode_step_token_gb300 import Sampler  # noqa: E402


class Micro:
    """A matrix in microscaled 4 bits, in buffers that are kept."""

    def __init__(self, sampler: Sampler, rows: int, cols: int, block: int, device):
        self.sampler, self.block, self.cols = sampler, block, cols
        self.values = torch.empty((rows, -(-cols // 32) * 16), dtype=torch.uint8, device=device)[:, :-(-cols // 2)]
        self.scales = torch.empty(sampler.micro_scale_bytes(rows, cols, block), dtype=torch.uint8, device=device)
        self.row_scale = torch.empty(rows, device=device)

    def lay_out(self, src: torch.Tensor) -> None:
        self.sampler.quantize_micro(src=src, out_values=self.values, out_scales=self.scales, out_row_scale=self.row_scale,
                                    block=self.block)

    def rows(self, out: torch.Tensor, ids: torch.Tensor = None) -> torch.Tensor:
        self.sampler.micro_rows(values=self.values, scales=self.scales, row_scale=self.row_scale, ids=ids, out=out,
                                block=self.block)
        return out

    def operand(self, name: str) -> dict:
        return {name: self.values, name + "_scale": self.scales, name + "_row_scale": self.row_scale}


class Lesson:
    """What a teacher says about hidden states, and a student's step towards it."""

    def __init__(self, sampler: Sampler, rows: int, vocab: int, top: int, device):
        self.sampler = sampler
        self.ids = torch.empty((rows, top), dtype=torch.int32, device=device)
        self.logprobs = torch.empty((rows, top), device=device)
        self.rest = torch.empty(rows, device=device)
        self.weight = torch.full((rows,), 1.0 / rows, device=device)
        self.loss, self.kl = torch.empty(1, device=device), torch.empty(rows, device=device)
        self.grad = torch.empty((rows, vocab), device=device)

    def hear(self, logits: torch.Tensor) -> None:
        self.sampler.score_top(logits=logits, top_n=self.ids.shape[1], out_top_ids=self.ids, out_top_logprobs=self.logprobs,
                               out_rest_logprob=self.rest)

    def step(self, hidden: torch.Tensor, student: torch.Tensor, token_coef: float) -> torch.Tensor:
        """The gradient by the student's weight [vocab, width]."""
        self.sampler.distill_loss(logits=hidden @ student.t(), teacher_ids=self.ids, teacher_logprobs=self.logprobs,
                                  teacher_rest=self.rest, tokens=self.ids[:, 0].contiguous(), token_coef=token_coef,
                                  weight=self.weight, out_loss=self.loss, out_kl=self.kl, out_grad=self.grad)
        return self.grad.t() @ hidden


def run(rows: int = 64, vocab: int = 4096, width: int = 256, top: int = 32, rounds: int = 8, tokens: int = 8,
        block: int = 16, seed: int = 0) -> dict:
    """The mean divergence before each step, and the tokens [tokens, rows] that the student then gives."""
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(seed)
    hidden = torch.randn((rows, width), generator=gen, device=dev)
    teacher = 2.0 * torch.randn((vocab, width), generator=gen, device=dev) / width ** 0.5
    student = 0.1 * torch.randn((vocab, width), generator=gen, device=dev) / width ** 0.5
    with Sampler(max_rows=rows, max_vocab=vocab) as sampler:
        lesson = Lesson(sampler, rows, vocab, top, dev)
        divergence = []
        for _ in range(rounds):
            lesson.hear(hidden @ teacher.t())
            student.sub_(4.0 * lesson.step(hidden, student, token_coef=0.1))
            divergence.append(lesson.kl.mean().item())

        served, state = Micro(sampler, vocab, width, block, dev), Micro(sampler, rows, width, block, dev)
        served.lay_out(student)
        now = hidden.to(torch.bfloat16)
        logits = torch.empty((rows, vocab), dtype=torch.bfloat16, device=dev)
        out = torch.empty((tokens, rows), dtype=torch.int32, device=dev)
        logprob = torch.empty((tokens, rows), device=dev)
        for t in range(tokens):
            state.lay_out(now)
            args = sampler.make_args(logits=logits, temperature=torch.full((rows,), 0.8, device=dev), out_tokens=out[t],
                                     philox_offset=t)
            sampler.lm_head_micro_sample_args(args, out_token_logprob=logprob[t], **state.operand("hidden"),
                                              **served.operand("weight"), block=block)
            served.rows(now, ids=out[t])
        torch.cuda.synchronize()
    return dict(divergence=divergence, tokens=out.cpu(), logprob=logprob.cpu())


if __name__ == "__main__":
    result = run()
    for r, x in enumerate(result["divergence"]):
        print(f"round {r}: divergence {x:.4f}")
    print("tokens of the first row:", result["tokens"][:, 0].tolist())
