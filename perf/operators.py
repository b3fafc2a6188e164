"""What the post-training and 8-bit operators are measured on.

A user who samples with this library has the logits of the tokens that were sampled, and trains
on them or scores them: the logprob and entropy of given tokens (`score`) and their gradient,
the clipped policy loss with its KL term and gradient, the preference loss over pairs of answers
with its gradient; and makes the logits with an LM head held in 8 bits (`lm_head_scaled`), whose
operands `quantize_blocks` lays out. Each case below runs one of these calls.

`run` computes an operator in its plain form where `own` is false (elementary torch operations in
32 bits, 64 where sums are long or a value decides which side of a border it is on), and through
`decode_step_token_gb300.Sampler` where it is true.
"""
import math

import torch

own = False

DEVICE = "cuda:0"
MAX_ROWS, MAX_VOCAB = 8192, 262144
MOST_VALUES = 4096 * 128000            # logits of the largest loss case
MOST_PRODUCTS = 4096 * 128000 * 4096   # multiply-adds of the largest LM head
E4M3_MAX = 448.0
FLOOR_MAX = 2.0 ** -100                # blocks whose largest magnitude is below this are scaled as if it were this
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # logprobs and entropies of one decode step's tokens under another model, at the vocabulary of the
        # framework's latency workload: a few rows, where latency counts
        dict(name="score decode step", op="score", n=32, vocab=151936, type="bf16", pad=0, kept=1.0, banned=0.0,
             heat=True, grad=False),
        # any other loss on the same logprobs: their gradient with an entropy term, fp32, rows that start anywhere
        dict(name="score gradient odd f32", op="score", n=517, vocab=40961, type="f32", pad=2, kept=0.8, banned=0.1,
             heat=True, grad=True),
        # one token's update: the smallest call
        dict(name="policy one row", op="policy", n=1, vocab=151936, type="bf16", pad=0, kept=1.0, banned=0.0,
             heat=False, kl=True, entropy=False, grad=True),
        # the last, odd part of a batch, with an entropy bonus; a tenth of the rows is padding
        dict(name="policy odd rows f32", op="policy", n=127, vocab=128000, type="f32", pad=0, kept=0.9, banned=0.2,
             heat=True, kl=True, entropy=True, grad=True),
        # a whole micro-batch of sampled answers
        dict(name="policy batch", op="policy", n=4096, vocab=128000, type="bf16", pad=0, kept=0.9, banned=0.0,
             heat=True, kl=True, entropy=False, grad=True),
        # a few short pairs over a small vocabulary: launches count
        dict(name="pairs short", op="pairs", pairs=4, longest=40, vocab=1024, type="f32", pad=0, kept=0.6,
             banned=0.0, per_token=False, grad=True),
        # pairs of answers after masked prompts at the headline vocabulary
        dict(name="pairs batch", op="pairs", pairs=8, longest=256, vocab=128000, type="bf16", pad=0, kept=0.7,
             banned=0.0, per_token=True, grad=True),
        # a decode step's hidden rows to 8 bits, one scale for 128 values
        dict(name="quantize hidden", op="quantize", rows=64, cols=4096, type="bf16", pad=0, square=False),
        # the LM head's weight to 8 bits, one scale for 128 x 128 values: once for each new weight
        dict(name="quantize weight", op="quantize", rows=128000, cols=4096, type="bf16", pad=0, square=True),
        # the headline step's LM head
        dict(name="head decode", op="head", rows=64, vocab=128000, k=4096, type="bf16"),
        # ragged in every direction, fp32 logits
        dict(name="head ragged f32", op="head", rows=333, vocab=20011, k=1000, type="f32"),
        # the logits of a prompt's tokens, for scoring
        dict(name="head prompt", op="head", rows=4096, vocab=128000, k=4096, type="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("score", "policy", "pairs", "quantize", "head"))
    kind = rng.choice(("bf16", "bf16", "f32"))
    if op == "quantize":
        rows = _spread(rng, 1, 128000)
        cols = min(_spread(rng, 128, 16384), 128000 * 4096 // rows)
        return dict(op=op, rows=rows, cols=cols, type=kind, pad=rng.choice((0, 0, 1, 8)), square=rng.random() < 0.5)
    if op == "head":
        rows, vocab = _spread(rng, 1, 4096), _spread(rng, 1000, 151936)
        k = min(_spread(rng, 64, 8192), MOST_PRODUCTS // (rows * vocab))
        return dict(op=op, rows=rows, vocab=vocab, k=k, type=kind)
    # a fp32 value counts for two: the largest case is in 16 bits
    most = MOST_VALUES // (BYTES[kind] // 2)
    vocab = _spread(rng, 500, 262144)
    rest = dict(type=kind, pad=rng.choice((0, 0, 1, 3, 8)), kept=rng.choice((1.0, 0.9, 0.5)),
                banned=rng.choice((0.0, 0.0, 0.3)), grad=rng.random() < 0.75)
    if op == "pairs":
        pairs = _spread(rng, 1, 32)
        longest = max(2, min(_spread(rng, 8, 512), most // (vocab * 2 * pairs), MAX_ROWS // (2 * pairs)))
        return dict(op=op, pairs=pairs, longest=longest, vocab=vocab, per_token=rng.random() < 0.5, **rest)
    n = _spread(rng, 1, max(1, min(4096, most // vocab)))
    if op == "score":
        return dict(op=op, n=n, vocab=vocab, heat=rng.random() < 0.5, **rest)
    return dict(op=op, n=n, vocab=vocab, heat=rng.random() < 0.5, kl=rng.random() < 0.7, entropy=rng.random() < 0.4,
                **rest)


# --------------------------------------------------------------------------- what a case's sizes are
def _lengths(case):
    """Rows of each of the 2 * pairs answers: between half of the longest and all of it."""
    longest = case["longest"]
    return [max(1, longest - (i * 7919) % max(1, longest // 2 + 1)) for i in range(2 * case["pairs"])]


def _rows(case):
    return sum(_lengths(case)) if case["op"] == "pairs" else case["n"]


def _kept(case):
    return max(1, round(case["kept"] * _rows(case)))


def _groups(n):
    return -(-n // 128)


# -------------------------------------------------------------------------------------- the inputs
_handle = None


def _sampler():
    """The library handle that a program creates once and keeps."""
    global _handle
    if _handle is None:
        from decode_step_token_gb300 import Sampler

        _handle = Sampler(max_rows=MAX_ROWS, max_vocab=MAX_VOCAB)
    return _handle


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    if case["op"] == "quantize":
        state = _prepare_quantize(case, gen)
    elif case["op"] == "head":
        state = _prepare_head(case, gen)
    else:
        state = _prepare_rows(case, gen)
    state["case"] = case
    if own:
        state["sampler"] = _sampler()
    return state


def _prepare_quantize(case, gen):
    rows, cols, es = case["rows"], case["cols"], BYTES[case["type"]]
    stride = cols + case["pad"]
    src = torch.randn((rows, stride), generator=gen, device=DEVICE, dtype=TYPES[case["type"]])
    # features of very different sizes, as hidden states and weights have them
    src.mul_(torch.exp(1.5 * torch.randn(stride, generator=gen, device=DEVICE)).to(src.dtype))
    src = src[:, :cols]
    if rows > 1:
        src[rows // 2].zero_()
    q_stride = -(-cols // 16) * 16
    scale_rows = _groups(rows) if case["square"] else rows
    return dict(src=src, values=torch.empty((rows, q_stride), dtype=torch.float8_e4m3fn, device=DEVICE)[:, :cols],
                scales=torch.empty((scale_rows, _groups(cols)), dtype=torch.float32, device=DEVICE))


def _prepare_head(case, gen):
    rows, vocab, k = case["rows"], case["vocab"], case["k"]
    stride = -(-k // 16) * 16

    def eight(n):
        # normal values, scaled so that a block's largest is near the type's largest
        x = torch.randn((n, stride), generator=gen, device=DEVICE, dtype=torch.bfloat16).mul_(100.0).clamp_(-448.0, 448.0)
        return x.to(torch.float8_e4m3fn)[:, :k]

    def scales(n, size):
        spread = torch.exp(0.5 * torch.randn((n, _groups(k)), generator=gen, device=DEVICE))
        return spread * (size / 100.0)

    return dict(hidden=eight(rows), hidden_scale=scales(rows, 1.0), weight=eight(vocab),
                weight_scale=scales(_groups(vocab), 2.0 / math.sqrt(k)),
                logits=torch.empty((rows, vocab), dtype=TYPES[case["type"]], device=DEVICE))


def _prepare_rows(case, gen):
    n, vocab, kind = _rows(case), case["vocab"], TYPES[case["type"]]
    stride = vocab + case["pad"]
    logits = torch.randn((n, stride), generator=gen, device=DEVICE, dtype=kind).mul_(2.0)[:, :vocab]
    rows = torch.arange(n, device=DEVICE)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=DEVICE)

    def normal(scale):
        return scale * torch.randn(n, generator=gen, device=DEVICE)

    # most sampled tokens are likely ones: their logit is 8 to 14
    tokens = torch.randint(0, vocab, (n,), generator=gen, device=DEVICE)
    likely = uniform(n) < 0.8
    at = logits[rows, tokens]
    logits[rows, tokens] = torch.where(likely, (8.0 + 6.0 * uniform(n)).to(kind), at)
    if case["banned"]:  # tokens that a grammar forbids, on some of the rows
        ban = torch.rand(vocab, generator=gen, device=DEVICE) < case["banned"]
        some = uniform(n) < 0.5
        keep = logits[rows, tokens]
        for r in torch.nonzero(some).flatten().tolist():
            logits[r].masked_fill_(ban, -math.inf)
        logits[rows, tokens] = keep
    state = dict(logits=logits, tokens=tokens.to(torch.int32), temperature=None)
    if case.get("heat"):
        state["temperature"] = 0.7 + 0.6 * uniform(n)
    # rows that are left out (padding, prompts): their logits are whatever was in the buffer
    m = _kept(case)
    weight = torch.zeros(n, device=DEVICE)
    order = torch.randperm(n, generator=gen, device=DEVICE)
    weight[order[:m]] = 1.0
    if m < n:
        logits[order[m:(m + n) // 2 + 1][:n - m]] = math.nan
    scale = state["temperature"] if state["temperature"] is not None else torch.ones(n, device=DEVICE)
    logprob = torch.empty(n, device=DEVICE)
    for a in range(0, n, 256):
        x = logits[a:a + 256].float() / scale[a:a + 256, None]
        logprob[a:a + 256] = x.gather(1, tokens[a:a + 256, None])[:, 0] - torch.logsumexp(x, 1)
    logprob = torch.where(weight > 0, logprob, 0.0)
    out = dict(logprob=torch.empty(n, device=DEVICE), entropy=torch.empty(n, device=DEVICE),
               loss=torch.empty(1, device=DEVICE))
    if case["grad"]:
        out["grad"] = torch.empty((n, stride), dtype=kind, device=DEVICE)[:, :vocab]
    if case["op"] == "score":
        state |= dict(weight=weight, grad_logprob=normal(1.0), grad_entropy=normal(0.1))
    elif case["op"] == "policy":
        state |= dict(weight=weight / m, old_logprob=logprob + normal(0.15), advantage=normal(1.0),
                      ref_logprob=logprob + normal(0.3) if case["kl"] else None)
        out |= dict(ratio=torch.empty(n, device=DEVICE), kl=torch.empty(n, device=DEVICE))
    else:
        offsets = [0]
        for length in _lengths(case):
            offsets.append(offsets[-1] + length)
        state |= dict(weight=weight, ref_logprob=logprob + normal(0.3),
                      seq_offsets=torch.tensor(offsets, dtype=torch.int32, device=DEVICE))
        out["reward"] = torch.empty(2 * case["pairs"], device=DEVICE)
    state["out"] = out
    return state


CLIP_LOW, CLIP_HIGH, KL_COEF, ENTROPY_COEF = 0.2, 0.28, 0.05, 0.01
BETA, MARGIN, SMOOTHING = 0.1, 0.0, 0.05
TOKEN_BETA, TOKEN_MARGIN = 2.0, 0.5   # of the form that takes each answer's mean over its tokens


def _pair_terms(case):
    return (TOKEN_BETA, TOKEN_MARGIN) if case["per_token"] else (BETA, MARGIN)


# ------------------------------------------------------------------------------------------- a pass
def run(state):
    op = state["case"]["op"]
    if op == "quantize":
        return _run_quantize(state)
    if op == "head":
        return _run_head(state)
    if op == "score":
        return _run_score(state)
    return _run_policy(state) if op == "policy" else _run_pairs(state)


def _run_quantize(state):
    square = state["case"]["square"]
    if own:
        state["sampler"].quantize_blocks(src=state["src"], block_rows=128 if square else 1,
                                         out_values=state["values"], out_scales=state["scales"])
        return dict(values=state["values"], scales=state["scales"])
    src = state["src"]
    rows, cols = src.shape
    height = 128 if square else 1
    up, across = -(-rows // height), _groups(cols)
    x = torch.zeros((up * height, across * 128), device=DEVICE)
    x[:rows, :cols] = src.float()
    x = x.view(up, height, across, 128)
    most = x.abs().amax(dim=(1, 3)).clamp(min=FLOOR_MAX)
    values = (x * (E4M3_MAX / most)[:, None, :, None]).to(torch.float8_e4m3fn)
    values = values.view(up * height, across * 128)[:rows, :cols]
    return dict(values=values, scales=most / E4M3_MAX)


def _run_head(state):
    if own:
        state["sampler"].lm_head_scaled(hidden=state["hidden"], hidden_scale=state["hidden_scale"],
                                        weight=state["weight"], weight_scale=state["weight_scale"],
                                        logits=state["logits"])
        return state["logits"]
    k, vocab = state["hidden"].shape[1], state["weight"].shape[0]
    hidden = state["hidden"].float() * state["hidden_scale"].repeat_interleave(128, 1)[:, :k]
    scale = state["weight_scale"].repeat_interleave(128, 0)[:vocab].repeat_interleave(128, 1)[:, :k]
    return (hidden @ (state["weight"].float() * scale).t()).to(state["logits"].dtype)


def _softmax_parts(state):
    """(x - max, exp of it, its sum, the tokens' logprobs in 64 bits, the rows that count) of the rows' scaled logits."""
    live = state["weight"] > 0
    x = torch.where(live[:, None], state["logits"].float(), 0.0)
    if state["temperature"] is not None:
        x = x / state["temperature"][:, None]
    x = x - x.amax(1, keepdim=True)
    e = torch.exp(x)
    s = e.sum(1)
    logprob = x.gather(1, state["tokens"].long()[:, None])[:, 0].double() - torch.log(s.double())
    return x, e, s, logprob, live


def _entropy(x, e, s):
    return torch.log(s.double()) - (e * x.clamp(min=-1e30)).sum(1).double() / s.double()


def _logits_grad(state, x, e, s, logprob, by_logprob, entropy, by_entropy):
    """The logits' gradient from the gradients by each row's logprob and entropy (None: none)."""
    p = e / s[:, None]
    by_logprob = by_logprob.float()
    g = -p * by_logprob[:, None]
    if by_entropy is not None:
        logp = x.clamp(min=-1e30) - torch.log(s)[:, None]
        g = g - p * (logp + entropy.float()[:, None]) * by_entropy.float()[:, None]
    token = state["tokens"].long()[:, None]
    g.scatter_add_(1, token, by_logprob[:, None])
    if state["temperature"] is not None:
        g = g / state["temperature"][:, None]
    g = torch.where((state["weight"] > 0)[:, None], g, 0.0)
    return g.to(state["logits"].dtype)


def _run_score(state):
    case, out = state["case"], state["out"]
    if own:
        rows = dict(logits=state["logits"], tokens=state["tokens"], temperature=state["temperature"],
                    weight=state["weight"], out_logprob=out["logprob"], out_entropy=out["entropy"])
        if not case["grad"]:
            state["sampler"].score(**rows)
            return dict(logprob=out["logprob"], entropy=out["entropy"])
        state["sampler"].score_grad(grad_logprob=state["grad_logprob"], grad_entropy=state["grad_entropy"],
                                    out_grad=out["grad"], **rows)
        return dict(logprob=out["logprob"], entropy=out["entropy"], grad=out["grad"])
    x, e, s, logprob, live = _softmax_parts(state)
    entropy = _entropy(x, e, s)
    got = dict(logprob=torch.where(live, logprob, 0.0).float(), entropy=torch.where(live, entropy, 0.0).float())
    if case["grad"]:
        got["grad"] = _logits_grad(state, x, e, s, logprob, state["grad_logprob"], entropy, state["grad_entropy"])
    return got


def _run_policy(state):
    case, out = state["case"], state["out"]
    kl_coef = KL_COEF if case["kl"] else 0.0
    entropy_coef = ENTROPY_COEF if case["entropy"] else 0.0
    if own:
        state["sampler"].policy_loss(
            logits=state["logits"], tokens=state["tokens"], temperature=state["temperature"], weight=state["weight"],
            old_logprob=state["old_logprob"], advantage=state["advantage"], ref_logprob=state["ref_logprob"],
            clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=kl_coef, entropy_coef=entropy_coef,
            out_loss=out["loss"], out_logprob=out["logprob"], out_ratio=out["ratio"],
            out_kl=out["kl"] if case["kl"] else None, out_entropy=out["entropy"] if case["entropy"] else None,
            out_grad=out.get("grad"))
        names = ["loss", "logprob", "ratio"] + ["kl"] * case["kl"] + ["entropy"] * case["entropy"]
        return {k: out[k] for k in names + ["grad"] * case["grad"]}
    x, e, s, logprob, live = _softmax_parts(state)
    weight, advantage = state["weight"].double(), state["advantage"].double()
    ratio = torch.exp(logprob - state["old_logprob"].double())
    clipped = ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH)
    term = -torch.minimum(ratio * advantage, clipped * advantage)
    outside = ((advantage > 0) & (ratio > 1.0 + CLIP_HIGH)) | ((advantage < 0) & (ratio < 1.0 - CLIP_LOW))
    by_logprob = torch.where(outside, 0.0, -ratio * advantage)
    got = dict(logprob=torch.where(live, logprob, 0.0).float(), ratio=torch.where(live, ratio, 0.0).float())
    if case["kl"]:
        d = state["ref_logprob"].double() - logprob
        kl = torch.expm1(d) - d
        term = term + kl_coef * kl
        by_logprob = by_logprob - kl_coef * torch.expm1(d)
        got["kl"] = torch.where(live, kl, 0.0).float()
    entropy, by_entropy = None, None
    if case["entropy"]:
        entropy = _entropy(x, e, s)
        term = term - entropy_coef * entropy
        by_entropy = -entropy_coef * weight
        got["entropy"] = torch.where(live, entropy, 0.0).float()
    got["loss"] = torch.where(live, weight * term, 0.0).sum().float()[None]
    if case["grad"]:
        got["grad"] = _logits_grad(state, x, e, s, logprob, weight * by_logprob, entropy, by_entropy)
    return got


def _run_pairs(state):
    case, out = state["case"], state["out"]
    beta, margin = _pair_terms(case)
    if own:
        state["sampler"].preference_loss(
            logits=state["logits"], tokens=state["tokens"], weight=state["weight"], seq_offsets=state["seq_offsets"],
            ref_logprob=state["ref_logprob"], beta=beta, margin=margin, label_smoothing=SMOOTHING,
            mean_over_tokens=case["per_token"], out_loss=out["loss"], out_logprob=out["logprob"],
            out_reward=out["reward"], out_grad=out.get("grad"))
        return {k: out[k] for k in ["loss", "logprob", "reward"] + ["grad"] * case["grad"]}
    x, e, s, logprob, live = _softmax_parts(state)
    weight, bounds = state["weight"].double(), state["seq_offsets"].long()

    def sums(v):  # of each answer's rows
        c = torch.cat((torch.zeros(1, dtype=torch.float64, device=DEVICE), torch.cumsum(v, 0)))
        return c[bounds[1:]] - c[bounds[:-1]]

    total = sums(torch.where(live, weight * (logprob - state["ref_logprob"].double()), 0.0))
    share = torch.ones_like(total)
    if case["per_token"]:
        count = sums(weight)
        share = torch.where(count > 0, 1.0 / count, 0.0)
    reward = beta * total * share
    z = reward[0::2] - reward[1::2] - margin
    log_sigmoid = torch.clamp(z, max=0.0) - torch.log1p(torch.exp(-z.abs()))
    pairs = case["pairs"]
    loss = (-(1.0 - SMOOTHING) * log_sigmoid - SMOOTHING * (log_sigmoid - z)).sum() / pairs
    got = dict(loss=loss.float()[None], logprob=torch.where(live, logprob, 0.0).float(), reward=reward.float())
    if case["grad"]:
        by_z = (torch.sigmoid(z) - (1.0 - SMOOTHING)) / pairs
        by_total = torch.stack((by_z, -by_z), 1).flatten() * beta * share
        rows = torch.arange(weight.shape[0], device=DEVICE)
        answer = torch.searchsorted(bounds[1:].contiguous(), rows, right=True)
        got["grad"] = _logits_grad(state, x, e, s, logprob, weight * by_total[answer], None, None)
    return got


# ------------------------------------------------------------------------------- what a pass has to do
def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        groups = (_groups(case["rows"]) if case["square"] else case["rows"]) * _groups(case["cols"])
        return {"bytes": n * (BYTES[case["type"]] + 1) + 4 * groups, "flops": 2 * n}
    if case["op"] == "head":
        rows, vocab, k = case["rows"], case["vocab"], case["k"]
        return {"bytes": (rows + vocab) * k + rows * vocab * BYTES[case["type"]] + 4 * _groups(k) * (rows + _groups(vocab)),
                "flops": 2 * rows * vocab * k}
    n, vocab, es = _rows(case), case["vocab"], BYTES[case["type"]]
    live = _kept(case)
    # the rows that count are read once, the gradient is written once (zeros for the others);
    # a logit costs a subtraction, an exponential, a sum; its gradient two products more
    return {"bytes": live * vocab * es + (n * vocab * es if case["grad"] else 0) + 24 * n,
            "flops": live * vocab * (3 + (2 if case["grad"] else 0))}


# ------------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_quantize(state)
    if case["op"] == "head":
        return _exact_head(state)
    return _exact_rows(state)


def _exact_quantize(state):
    src, square = state["src"].double(), state["case"]["square"]
    values, scales = torch.empty_like(src), torch.empty(state["scales"].shape, dtype=torch.float64, device=DEVICE)
    height = 128 if square else src.shape[0]
    for j in range(scales.shape[1]):
        for i in range(0, src.shape[0], height):
            block = src[i:i + height, 128 * j:128 * j + 128]
            most = block.abs().max() if square else block.abs().max(1).values
            scale = torch.clamp(most, min=FLOOR_MAX) / E4M3_MAX
            at = i // 128 if square else slice(None)
            scales[at, j] = scale
            values[i:i + height, 128 * j:128 * j + 128] = _nearest_e4m3(block / (scale if square else scale[:, None]))
    return dict(values=values, scales=scales)


def _nearest_e4m3(x):
    """The nearest number of 4 significant bits whose exponent is -6 or more, up to 448; ties to even."""
    _, exponent = torch.frexp(x.abs().clamp(min=2.0 ** -6))
    step = torch.ldexp(torch.ones_like(x), exponent - 4)
    return torch.clamp(torch.round(x / step) * step, -E4M3_MAX, E4M3_MAX)


def _exact_head(state):
    rows, k = state["hidden"].shape
    vocab = state["weight"].shape[0]
    out = torch.zeros((rows, vocab), dtype=torch.float64, device=DEVICE)
    for b in range(0, k, 128):
        h = state["hidden"][:, b:b + 128].double() * state["hidden_scale"][:, b // 128].double()[:, None]
        w = state["weight"][:, b:b + 128].double()
        w.mul_(state["weight_scale"][:, b // 128].double().repeat_interleave(128)[:vocab, None])
        out.addmm_(h, w.t())
    return out


def _exact_rows(state):
    case, n = state["case"], state["logits"].shape[0]
    weight, tokens = state["weight"].double(), state["tokens"].long()
    logprob = torch.zeros(n, dtype=torch.float64, device=DEVICE)
    entropy = torch.zeros_like(logprob)

    def some(a, b):
        """The rows a..b that count, their scaled logits in 64 bits, and from those their logprobs and entropies."""
        at = a + torch.nonzero(weight[a:b] > 0).flatten()
        x = state["logits"][at].double().requires_grad_(case["grad"])
        scaled = x if state["temperature"] is None else x / state["temperature"][at].double()[:, None]
        logp = torch.log_softmax(scaled, 1)
        # a forbidden token has no share in the entropy
        h = -torch.where(logp > -math.inf, torch.exp(logp) * torch.where(logp > -math.inf, logp, 0.0), 0.0).sum(1)
        return at, x, logp.gather(1, tokens[at, None])[:, 0], h

    step = max(1, (64 << 20) // case["vocab"])
    with torch.no_grad():
        for a in range(0, n, step):
            at, _, lp, h = some(a, a + step)
            logprob[at], entropy[at] = lp, h
    live = weight > 0
    lp, h = logprob.clone().requires_grad_(True), entropy.clone().requires_grad_(True)
    got = dict(logprob=logprob)
    if case["op"] == "score":
        got["entropy"] = entropy
        target = (lp * state["grad_logprob"].double() + h * state["grad_entropy"].double())[live].sum()
    elif case["op"] == "policy":
        ratio = torch.exp(lp - state["old_logprob"].double())
        advantage = state["advantage"].double()
        gain = torch.minimum(ratio * advantage, ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * advantage)
        each = -gain
        got["ratio"] = torch.where(live, ratio, 0.0).detach()
        if case["kl"]:
            d = state["ref_logprob"].double() - lp
            each = each + KL_COEF * (torch.expm1(d) - d)
            got["kl"] = torch.where(live, torch.expm1(d) - d, 0.0).detach()
        if case["entropy"]:
            each = each - ENTROPY_COEF * h
            got["entropy"] = entropy
        target = (each * weight)[live].sum()
        got["loss"] = target.detach()[None]
    else:
        beta, margin = _pair_terms(case)
        ends = state["seq_offsets"].tolist()
        rewards = []
        for a, b in zip(ends[:-1], ends[1:]):
            r = (weight[a:b] * (lp[a:b] - state["ref_logprob"][a:b].double())).sum()
            if case["per_token"]:
                r = r / weight[a:b].sum() if float(weight[a:b].sum()) > 0 else r * 0.0
            rewards.append(beta * r)
        z = torch.stack(rewards[0::2]) - torch.stack(rewards[1::2]) - margin
        sure = torch.nn.functional.logsigmoid
        target = (-(1.0 - SMOOTHING) * sure(z) - SMOOTHING * sure(-z)).mean()
        got |= dict(loss=target.detach()[None], reward=torch.stack(rewards).detach())
    if case["grad"]:
        by = torch.autograd.grad(target, (lp, h), allow_unused=True)
        by = [torch.zeros_like(lp) if v is None else v for v in by]
        grad = torch.zeros((n, case["vocab"]), dtype=torch.float64, device=DEVICE)
        for a in range(0, n, step):
            at, x, lp_here, h_here = some(a, a + step)
            ends = [lp_here, h_here] if bool(by[1].abs().sum() > 0) else [lp_here]
            grad[at] = torch.autograd.grad(ends, x, [v[at] for v in by[:len(ends)]])[0]
        got["grad"] = grad
    return got
