"""What the distillation and 4-bit operators are measured on.

A user who samples with this library distils from the model that they sample: the teacher's rows give their most
likely tokens with the logprob of the rest (`score_top`), and the student's rows the loss against those and its
gradient (`distill_loss`). What is trained that way is served with an LM head in microscaled 4 bits
(`lm_head_micro`), whose operands `quantize_micro` lays out and `micro_rows` reads back. Each case below runs one of
these, the quantiser with its reading back.

`run` computes an operator in its plain form where `own` is false (elementary torch operations in 32 bits, 64 where
sums are long or cancel), and through `decode_step_token_gb300.Sampler` where it is true.
"""
import math

import torch

own = False

DEVICE = "cuda:0"
MAX_ROWS, MAX_VOCAB = 8192, 262144
MOST_VALUES = 4096 * 128000            # 16-bit logits of the largest case over rows
MOST_PRODUCTS = 4096 * 128000 * 4096   # multiply-adds of the largest LM head
MOST_TOP = 128
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # the most likely tokens of one decode step's rows with their logprobs, beside the sampled tokens' own, at the
        # vocabulary of the framework's latency workload: latency counts
        dict(name="top decode step", op="top", n=32, vocab=151936, top=20, type="bf16", pad=0, kept=1.0, banned=0.0,
             heat=True, tokens=True, entropy=False),
        # fp32 rows that start anywhere, as many alternatives as there may be, tokens that a grammar forbids, entropies
        dict(name="top odd f32", op="top", n=517, vocab=40961, top=128, type="f32", pad=2, kept=0.8, banned=0.1,
             heat=True, tokens=True, entropy=True),
        # the teacher's pass over a micro-batch of answers: 64 tokens of each row and the mass of the rest
        dict(name="top teacher batch", op="top", n=4096, vocab=128000, top=64, type="bf16", pad=0, kept=0.9,
             banned=0.0, heat=False, tokens=False, entropy=False),
        # a few rows over a small vocabulary: launches count
        dict(name="distil few rows", op="distil", n=4, vocab=1024, top=8, type="f32", pad=0, kept=1.0, heat=False,
             rest=True, token=0.0, short=0.0, grad=True),
        # the last, odd part of a batch in fp32 with a share of the tokens' own loss; lists of different lengths
        dict(name="distil odd rows f32", op="distil", n=127, vocab=128000, top=100, type="f32", pad=0, kept=0.9,
             heat=True, rest=False, token=0.3, short=0.5, grad=True),
        # a whole micro-batch against the teacher's pass above
        dict(name="distil batch", op="distil", n=4096, vocab=128000, top=64, type="bf16", pad=0, kept=0.9, heat=False,
             rest=True, token=0.1, short=0.0, grad=True),
        # a decode step's hidden rows to 4 bits and back
        dict(name="micro hidden", op="micro", rows=64, cols=4096, type="bf16", pad=0, block=16),
        # the LM head's weight to 4 bits and back: once for each new weight
        dict(name="micro weight", op="micro", rows=128000, cols=4096, type="bf16", pad=0, block=32),
        # one token of a small model: the smallest product
        dict(name="head one token", op="head", rows=1, vocab=151936, k=2048, type="bf16", block=32),
        # the headline step's LM head
        dict(name="head decode", op="head", rows=64, vocab=128000, k=4096, type="bf16", block=16),
        # ragged in every direction, fp32 logits
        dict(name="head ragged f32", op="head", rows=333, vocab=20011, k=1000, type="f32", block=32),
        # the logits of a prompt's tokens, for scoring
        dict(name="head prompt", op="head", rows=4096, vocab=128000, k=4096, type="bf16", block=16),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("top", "distil", "micro", "head"))
    kind = rng.choice(("bf16", "bf16", "f32"))
    if op == "micro":
        rows = _spread(rng, 1, 128000)
        cols = min(_spread(rng, 64, 16384), 128000 * 4096 * 2 // (rows * BYTES[kind]))
        return dict(op=op, rows=rows, cols=cols, type=kind, pad=rng.choice((0, 0, 1, 8)), block=rng.choice((16, 32)))
    if op == "head":
        rows, vocab = _spread(rng, 1, 4096), _spread(rng, 1000, 151936)
        k = min(_spread(rng, 64, 8192), MOST_PRODUCTS // (rows * vocab))
        return dict(op=op, rows=rows, vocab=vocab, k=k, type=kind, block=rng.choice((16, 32)))
    vocab = _spread(rng, 500, 262144)
    # a fp32 value counts for two: the largest case is in 16 bits
    n = _spread(rng, 1, max(1, min(4096, MOST_VALUES // (BYTES[kind] // 2) // vocab)))
    rest = dict(n=n, vocab=vocab, top=_spread(rng, 1, MOST_TOP), type=kind, pad=rng.choice((0, 0, 1, 3, 8)),
                kept=rng.choice((1.0, 0.9, 0.5)), heat=rng.random() < 0.5)
    if op == "top":
        return dict(op=op, banned=rng.choice((0.0, 0.0, 0.3)), tokens=rng.random() < 0.5, entropy=rng.random() < 0.3,
                    **rest)
    return dict(op=op, rest=rng.random() < 0.6, token=rng.choice((0.0, 0.1, 0.5)), short=rng.choice((0.0, 0.0, 0.5)),
                grad=rng.random() < 0.8, **rest)


# --------------------------------------------------------------------------- what a case's sizes are
def _kept(case):
    return max(1, round(case["kept"] * case["n"]))


def _groups(n, size):
    return -(-n // size)


def _scale_tiles(rows, cols, block):
    """Tiles of 128 rows by 4 blocks that hold the scales."""
    return _groups(rows, 128), _groups(_groups(cols, block), 4)


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
    state = {"top": _prepare_top, "distil": _prepare_distil, "micro": _prepare_micro, "head": _prepare_head}[
        case["op"]](case, gen)
    state["case"] = case
    if own:
        state["sampler"] = _sampler()
    return state


def _uniform(gen, *shape):
    return torch.rand(shape, generator=gen, device=DEVICE)


def _logits(case, gen):
    """Rows of normal logits with a likely token on most of them, and those tokens."""
    n, vocab, kind = case["n"], case["vocab"], TYPES[case["type"]]
    stride = vocab + case["pad"]
    logits = torch.randn((n, stride), generator=gen, device=DEVICE, dtype=kind).mul_(2.0)[:, :vocab]
    rows = torch.arange(n, device=DEVICE)
    tokens = torch.randint(0, vocab, (n,), generator=gen, device=DEVICE)
    likely = _uniform(gen, n) < 0.8
    at = logits[rows, tokens]
    logits[rows, tokens] = torch.where(likely, (8.0 + 6.0 * _uniform(gen, n)).to(kind), at)
    return logits, tokens


def _weights(case, gen, logits):
    """1 for the rows that count, 0 for the others, whose logits are whatever was in the buffer."""
    n, m = case["n"], _kept(case)
    weight = torch.zeros(n, device=DEVICE)
    order = torch.randperm(n, generator=gen, device=DEVICE)
    weight[order[:m]] = 1.0
    logits[order[m:]] = math.nan
    return weight


def _prepare_top(case, gen):
    n, vocab, top = case["n"], case["vocab"], case["top"]
    logits, tokens = _logits(case, gen)
    if case["banned"]:  # tokens that a grammar forbids, on half of the rows
        ban = _uniform(gen, vocab) < case["banned"]
        keep = logits[torch.arange(n, device=DEVICE), tokens]
        logits[::2].masked_fill_(ban[None], -math.inf)
        logits[torch.arange(n, device=DEVICE), tokens] = keep
    state = dict(logits=logits, weight=_weights(case, gen, logits), tokens=tokens.to(torch.int32) if case["tokens"] else None,
                 temperature=0.7 + 0.6 * _uniform(gen, n) if case["heat"] else None)
    out = dict(ids=torch.empty((n, top), dtype=torch.int32, device=DEVICE), logprobs=torch.empty((n, top), device=DEVICE),
               rest=torch.empty(n, device=DEVICE))
    if case["tokens"]:
        out["logprob"] = torch.empty(n, device=DEVICE)
    if case["entropy"]:
        out["entropy"] = torch.empty(n, device=DEVICE)
    state["out"] = out
    return state


def _prepare_distil(case, gen):
    n, vocab, top, kind = case["n"], case["vocab"], case["top"], TYPES[case["type"]]
    logits, tokens = _logits(case, gen)
    state = dict(temperature=0.7 + 0.6 * _uniform(gen, n) if case["heat"] else None, tokens=tokens.to(torch.int32))
    # the teacher's rows are the student's with other values around them; its lists are its largest, of which some
    # rows have only the first few, and the mass of what is not in the list
    ids = torch.empty((n, top), dtype=torch.int32, device=DEVICE)
    logprobs, rest = torch.full((n, top), -math.inf, device=DEVICE), torch.empty(n, device=DEVICE)
    most = min(top, vocab)
    for a in range(0, n, 256):
        x = logits[a:a + 256].float()
        x = x + torch.randn(x.shape, generator=gen, device=DEVICE)
        if state["temperature"] is not None:
            x = x / state["temperature"][a:a + 256, None]
        x = x - torch.logsumexp(x, 1, keepdim=True)
        best, at = torch.topk(x, most, dim=1)
        count = torch.full((x.shape[0],), most, device=DEVICE)
        if case["short"]:
            fewer = 1 + (_uniform(gen, x.shape[0]) * most).long().clamp(max=most - 1)
            count = torch.where(_uniform(gen, x.shape[0]) < case["short"], fewer, count)
        in_list = torch.arange(most, device=DEVICE)[None] < count[:, None]
        ids[a:a + 256] = -1
        ids[a:a + 256, :most] = torch.where(in_list, at, -1).int()
        logprobs[a:a + 256, :most] = torch.where(in_list, best, -math.inf)
        x.scatter_(1, at, torch.where(in_list, -math.inf, best))
        rest[a:a + 256] = torch.logsumexp(x, 1)
    state |= dict(ids=ids, logprobs=logprobs, rest=rest if case["rest"] else None, logits=logits)
    state["weight"] = _weights(case, gen, logits) / _kept(case)
    out = dict(loss=torch.empty(1, device=DEVICE), kl=torch.empty(n, device=DEVICE))
    if case["grad"]:
        out["grad"] = torch.empty((n, vocab + case["pad"]), dtype=kind, device=DEVICE)[:, :vocab]
    state["out"] = out
    return state


def _prepare_micro(case, gen):
    rows, cols, kind, block = case["rows"], case["cols"], TYPES[case["type"]], case["block"]
    stride = cols + case["pad"]
    src = torch.randn((rows, stride), generator=gen, device=DEVICE, dtype=kind)
    # features of very different sizes, as hidden states and weights have them
    src.mul_(torch.exp(1.5 * torch.randn(stride, generator=gen, device=DEVICE)).to(kind))
    src = src[:, :cols]
    if rows > 1:
        src[rows // 2].zero_()
    half = _groups(cols, 2)
    up, across = _scale_tiles(rows, cols, block)
    return dict(src=src, values=torch.empty((rows, _groups(half, 16) * 16), dtype=torch.uint8, device=DEVICE)[:, :half],
                scales=torch.empty(up * across * 512, dtype=torch.uint8, device=DEVICE),
                row_scale=torch.empty(rows, device=DEVICE), back=torch.empty((rows, cols), dtype=kind, device=DEVICE))


def _prepare_head(case, gen):
    rows, vocab, k, block = case["rows"], case["vocab"], case["k"], case["block"]
    half = _groups(k, 2)

    def codes(n):
        # e2m1 codes of normal values scaled so that a block's largest is near the type's largest, two to a byte
        x = torch.randn((n, 2 * half), generator=gen, device=DEVICE).mul_(2.5)
        if k % 2:
            x[:, -1] = 0.0
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEVICE)
        c = (torch.bucketize(x.abs(), edges, out_int32=True) + 8 * (x < 0)).to(torch.uint8)
        values = torch.zeros((n, _groups(half, 16) * 16), dtype=torch.uint8, device=DEVICE)
        values[:, :half] = c[:, 0::2] | (c[:, 1::2] << 4)
        return values[:, :half]

    def scales(n):
        up, across = _scale_tiles(n, k, block)
        # e4m3 from 2^-2 to 15, or powers of two from 2^-4 to 2^3; tiles are padded with zeros
        lo, hi = (0x28, 0x57) if block == 16 else (123, 131)
        s = torch.randint(lo, hi, (up, across, 32, 4, 4), generator=gen, device=DEVICE, dtype=torch.uint8)
        b = torch.arange(4 * across, device=DEVICE).view(1, across, 1, 1, 4)
        return torch.where(b < _groups(k, block), s, 0).to(torch.uint8).flatten()

    def row_scale(n, size):
        if block == 32:  # a power of two for each block needs none for the row
            return None
        return torch.exp(0.3 * torch.randn(n, generator=gen, device=DEVICE)) * size

    return dict(hidden=codes(rows), hidden_scale=scales(rows), hidden_row_scale=row_scale(rows, 0.1),
                weight=codes(vocab), weight_scale=scales(vocab), weight_row_scale=row_scale(vocab, 0.1 / math.sqrt(k)),
                logits=torch.empty((rows, vocab), dtype=TYPES[case["type"]], device=DEVICE))


# ------------------------------------------------------------------------------------------- a pass
def run(state):
    return {"top": _run_top, "distil": _run_distil, "micro": _run_micro, "head": _run_head}[state["case"]["op"]](state)


def _scaled(state):
    """(x - max, exp of it, its sum, the largest x, the rows that count) of the rows' scaled logits."""
    live = state["weight"] > 0
    x = torch.where(live[:, None], state["logits"].float(), 0.0)
    if state["temperature"] is not None:
        x = x / state["temperature"][:, None]
    x = x - x.amax(1, keepdim=True)
    e = torch.exp(x)
    return x, e, e.sum(1), live


def _run_top(state):
    case, out = state["case"], state["out"]
    top, vocab = case["top"], case["vocab"]
    if own:
        state["sampler"].score_top(
            logits=state["logits"], top_n=top, tokens=state["tokens"], temperature=state["temperature"],
            weight=state["weight"], out_top_ids=out["ids"], out_top_logprobs=out["logprobs"], out_rest_logprob=out["rest"],
            out_logprob=out.get("logprob"), out_entropy=out.get("entropy"))
        return dict(out)
    x, e, s, live = _scaled(state)
    # largest value first, the lowest token first among equal ones: one whole number for both, as float bits in order
    raw = torch.where(live[:, None], state["logits"].float() + 0.0, 0.0)
    bits = raw.view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long()
    key = order * (1 << 18) + (vocab - 1 - torch.arange(vocab, device=DEVICE))[None]
    most = min(top, vocab)
    at = vocab - 1 - (torch.topk(key, most, dim=1).values & ((1 << 18) - 1))
    log_s = torch.log(s.double())
    best = x.gather(1, at).double() - log_s[:, None]
    some = best > -math.inf
    e_rest = e.scatter(1, at, 0.0)
    rest = torch.log(e_rest.sum(1).double()) - log_s
    ids = torch.full((case["n"], top), -1, dtype=torch.int32, device=DEVICE)
    logprobs = torch.full((case["n"], top), -math.inf, device=DEVICE)
    ids[:, :most] = torch.where(some & live[:, None], at, -1).int()
    logprobs[:, :most] = best.float()
    got = dict(ids=ids, logprobs=torch.where(live[:, None], logprobs, 0.0), rest=torch.where(live, rest, 0.0).float())
    if case["tokens"]:
        lp = x.gather(1, state["tokens"].long()[:, None])[:, 0].double() - log_s
        got["logprob"] = torch.where(live, lp, 0.0).float()
    if case["entropy"]:
        h = log_s - (e * x.clamp(min=-1e30)).sum(1).double() / s.double()
        got["entropy"] = torch.where(live, h, 0.0).float()
    return got


def _run_distil(state):
    case, out = state["case"], state["out"]
    if own:
        state["sampler"].distill_loss(
            logits=state["logits"], teacher_ids=state["ids"], teacher_logprobs=state["logprobs"],
            teacher_rest=state["rest"], tokens=state["tokens"] if case["token"] else None, token_coef=case["token"],
            temperature=state["temperature"], weight=state["weight"], out_loss=out["loss"], out_kl=out["kl"],
            out_grad=out.get("grad"))
        return dict(out)
    n, vocab = case["n"], case["vocab"]
    x, e, _, live = _scaled(state)
    # a divergence is a small difference of logprobs: sums, and the logits that it is made of, in 64 bits
    s = e.sum(1, dtype=torch.float64)
    weight, log_s = state["weight"].double(), torch.log(s)
    heat = torch.ones(n, device=DEVICE) if state["temperature"] is None else state["temperature"]
    most = torch.where(live, state["logits"].amax(1).double(), 0.0)

    def logprob(at):
        z = torch.where(live[:, None], state["logits"].gather(1, at).double(), 0.0)
        return (z - most[:, None]) / heat.double()[:, None] - log_s[:, None]

    ids = state["ids"].long()
    listed_ = ids >= 0
    bin_ = torch.where(listed_, ids, vocab)  # entries that are not there go to a column of their own
    e_rest = torch.cat((e, torch.zeros((n, 1), device=DEVICE)), 1)
    e_list = e_rest.gather(1, bin_)
    e_rest.scatter_(1, bin_, 0.0)
    teacher = state["logprobs"].double()
    q = torch.where(listed_, torch.exp(teacher), 0.0)
    mine = logprob(torch.where(listed_, ids, 0))
    kl = torch.where(q > 0, q * (teacher - mine), 0.0).sum(1)
    total = q.sum(1)
    by_rest = torch.zeros(n, dtype=torch.float64, device=DEVICE)
    if case["rest"]:
        r = state["rest"].double()
        qr = torch.exp(r)
        s_rest = e_rest.sum(1, dtype=torch.float64)
        kl = kl + torch.where(qr > 0, qr * (r - torch.log(s_rest) + log_s), 0.0)
        total = total + qr
        by_rest = torch.where(s_rest > 0, qr / s_rest, 0.0)  # of each exponential outside the list
    token = state["tokens"].long()[:, None]
    each = kl
    if case["token"]:
        each = kl - case["token"] * logprob(token)[:, 0]
        total = total + case["token"]
    got = dict(loss=torch.where(live, weight * each, 0.0).sum().float()[None], kl=torch.where(live, kl, 0.0).float())
    if case["grad"]:
        scale = weight / heat.double()
        g = e_rest * ((total / s - by_rest) * scale).float()[:, None]
        g.scatter_add_(1, bin_, e_list * (total / s * scale).float()[:, None] - (q * scale[:, None]).float())
        if case["token"]:
            g.scatter_add_(1, token, (-case["token"] * scale).float()[:, None])
        got["grad"] = torch.where(live[:, None], g[:, :vocab], 0.0).to(state["logits"].dtype)
    return got


def _run_micro(state):
    block = state["case"]["block"]
    if own:
        s = state["sampler"]
        s.quantize_micro(src=state["src"], block=block, out_values=state["values"], out_scales=state["scales"],
                         out_row_scale=state["row_scale"])
        s.micro_rows(values=state["values"], scales=state["scales"], row_scale=state["row_scale"], block=block,
                     out=state["back"])
        return dict(back=state["back"], row_scale=state["row_scale"])
    src = state["src"]
    rows, cols = src.shape
    across = _groups(cols, block)
    x = torch.zeros((rows, across * block), device=DEVICE)
    x[:, :cols] = src.float()
    x = x.view(rows, across, block)
    most = x.abs().amax(2)

    def least_power(m, sixth):
        """The exponent of the least power of two whose `sixth` (1 to 2, of 2^0) multiple is m or more."""
        bits = m.view(torch.int32)
        return (bits >> 23) - 127 + ((bits & 0x7fffff) > int((sixth - 1) * (1 << 23))).int()

    def power(e):
        return torch.where(e >= -126, ((e + 127).clamp(min=0) << 23), 1 << 22).view(torch.float32)

    if block == 32:
        row_scale = torch.ones(rows, device=DEVICE)
        scale = power((least_power(most, 1.5) - 2).clamp(min=-127))
    else:
        row_scale = power(least_power(most.amax(1).clamp(min=2.0 ** -100), 1.3125) - 11)
        sixth = most / torch.full_like(most, 6.0) / row_scale[:, None]
        scale = sixth.to(torch.float8_e4m3fn).float()
    unit = (scale * row_scale[:, None])[:, :, None]
    a = (x / torch.where(unit > 0, unit, 1.0)).abs().clamp(max=6.0)
    a = torch.where(unit > 0, a, 0.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    back = torch.copysign(torch.round(a / step) * step, x) * unit
    return dict(back=back.view(rows, across * block)[:, :cols].to(src.dtype), row_scale=row_scale)


def _run_head(state):
    case = state["case"]
    if own:
        state["sampler"].lm_head_micro(
            hidden=state["hidden"], hidden_scale=state["hidden_scale"], hidden_row_scale=state["hidden_row_scale"],
            weight=state["weight"], weight_scale=state["weight_scale"], weight_row_scale=state["weight_row_scale"],
            hidden_dim=case["k"], block=case["block"], logits=state["logits"])
        return state["logits"]
    k, block = case["k"], case["block"]
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=DEVICE)

    def values(packed, scales, row_scale):
        n = packed.shape[0]
        x = torch.stack((table[(packed & 15).int()], table[(packed >> 4).int()]), 2).view(n, -1)[:, :k]
        up, across = _scale_tiles(n, k, block)
        s = scales.view(up, across, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(up * 128, across * 4)[:n]
        s = s.contiguous().view(torch.float8_e4m3fn).float() if block == 16 else (s.int() << 23).view(torch.float32)
        if row_scale is not None:
            s = s * row_scale[:, None]
        return x * s.repeat_interleave(block, 1)[:, :k]

    hidden = values(state["hidden"], state["hidden_scale"], state["hidden_row_scale"])
    weight = values(state["weight"], state["weight_scale"], state["weight_row_scale"])
    return (hidden @ weight.t()).to(state["logits"].dtype)


# ------------------------------------------------------------------------------- what a pass has to do
def work(case):
    es = BYTES[case["type"]]
    if case["op"] == "micro":
        n, block = case["rows"] * case["cols"], case["block"]
        # the source once, the codes with their scales out and in, the values once
        held = n // 2 + case["rows"] * (_groups(case["cols"], block) + 4)
        return {"bytes": 2 * n * es + 2 * held, "flops": 4 * n}
    if case["op"] == "head":
        rows, vocab, k, block = case["rows"], case["vocab"], case["k"], case["block"]
        held = (rows + vocab) * (_groups(k, 2) + _groups(k, block) + (4 if block == 16 else 0))
        return {"bytes": held + rows * vocab * es, "flops": 2 * rows * vocab * k}
    n, vocab, live = case["n"], case["vocab"], _kept(case)
    # the rows that count are read once, the gradient is written once (zeros for the others); a logit costs a
    # subtraction, an exponential, a sum; its gradient two products more, its place in the order a comparison
    if case["op"] == "top":
        return {"bytes": live * vocab * es + n * (8 * case["top"] + 16), "flops": live * vocab * 4}
    return {"bytes": live * vocab * es + (n * vocab * es if case["grad"] else 0) + n * (8 * case["top"] + 16),
            "flops": live * vocab * (3 + (2 if case["grad"] else 0))}


# ------------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    return {"top": _exact_top, "distil": _exact_distil, "micro": _exact_micro, "head": _exact_head}[case["op"]](state)


def _row_steps(state):
    """(rows that count, their log probabilities in 64 bits with their logits as leaves) some rows at a time."""
    n, vocab = state["logits"].shape
    step = max(1, (64 << 20) // vocab)
    live = torch.nonzero(state["weight"] > 0).flatten()
    for a in range(0, live.numel(), step):
        at = live[a:a + step]
        x = state["logits"][at].double().requires_grad_(True)
        z = x if state["temperature"] is None else x / state["temperature"][at].double()[:, None]
        yield at, x, torch.log_softmax(z, 1)


def _exact_top(state):
    case = state["case"]
    n, top = case["n"], case["top"]
    got = dict(ids=torch.full((n, top), -1, dtype=torch.int32, device=DEVICE),
               logprobs=torch.zeros((n, top), dtype=torch.float64, device=DEVICE),
               rest=torch.zeros(n, dtype=torch.float64, device=DEVICE))
    if case["tokens"]:
        got["logprob"] = torch.zeros_like(got["rest"])
    if case["entropy"]:
        got["entropy"] = torch.zeros_like(got["rest"])
    with torch.no_grad():
        for at, x, logp in _row_steps(state):
            # a stable sort keeps equal logits in the order of their tokens
            best, order = torch.sort(x, dim=1, descending=True, stable=True)
            order, best = order[:, :top], best[:, :top]
            m = order.shape[1]
            got["logprobs"][at] = -math.inf
            got["logprobs"][at, :m] = logp.gather(1, order)
            got["ids"][at, :m] = torch.where(best > -math.inf, order, -1).int()
            got["rest"][at] = torch.logsumexp(logp.scatter(1, order, -math.inf), 1)
            if case["tokens"]:
                got["logprob"][at] = logp.gather(1, state["tokens"][at].long()[:, None])[:, 0]
            if case["entropy"]:
                got["entropy"][at] = -torch.where(logp > -math.inf, torch.exp(logp) * logp, 0.0).sum(1)
    return got


def _exact_distil(state):
    case = state["case"]
    n, vocab = case["n"], case["vocab"]
    weight = state["weight"].double()
    kl_all = torch.zeros(n, dtype=torch.float64, device=DEVICE)
    grad = torch.zeros((n, vocab), dtype=torch.float64, device=DEVICE) if case["grad"] else None
    loss = torch.zeros(1, dtype=torch.float64, device=DEVICE)
    for at, x, logp in _row_steps(state):
        ids, teacher = state["ids"][at].long(), state["logprobs"][at].double()
        there = ids >= 0
        mine = logp.gather(1, ids.clamp(min=0))
        kl = torch.where(there, torch.exp(teacher) * (torch.where(there, teacher, 0.0) - mine), 0.0).sum(1)
        if case["rest"]:
            inside = torch.zeros(logp.shape, dtype=torch.int32, device=DEVICE)
            inside.scatter_add_(1, ids.clamp(min=0), there.int())
            outside = torch.logsumexp(torch.where(inside > 0, -math.inf, logp), 1)
            r = state["rest"][at].double()
            some = (r > -math.inf) & (outside > -math.inf)
            kl = kl + torch.where(some, torch.exp(r) * (torch.where(some, r, 0.0) - torch.where(some, outside, 0.0)), 0.0)
        each = kl
        if case["token"]:
            each = kl - case["token"] * logp.gather(1, state["tokens"][at].long()[:, None])[:, 0]
        kl_all[at] = kl.detach()
        mean = (weight[at] * each).sum()
        loss += mean.detach()
        if grad is not None:
            grad[at] = torch.autograd.grad(mean, x)[0]
    got = dict(loss=loss, kl=kl_all)
    if grad is not None:
        got["grad"] = grad
    return got


def _exact_micro(state):
    src, block = state["src"], state["case"]["block"]
    rows, cols = src.shape
    back = torch.empty((rows, cols), dtype=torch.float64, device=DEVICE)
    row_scale = torch.ones(rows, dtype=torch.float64, device=DEVICE)
    for a in range(0, rows, 8192):
        x = src[a:a + 8192].double()
        if block == 16:
            # the least power of two of which the largest value is at most 448 * 6
            f, e = torch.frexp(x.abs().amax(1).clamp(min=2.0 ** -100) / 2688.0)
            row_scale[a:a + 8192] = _power(torch.where(f == 0.5, e - 1, e))
        for b in range(0, cols, block):
            y = x[:, b:b + block]
            sixth = y.abs().amax(1) / 6.0
            if block == 16:
                unit = _nearest(sixth / row_scale[a:a + 8192], 4, -6) * row_scale[a:a + 8192]
            else:
                f, e = torch.frexp(sixth.clamp(min=2.0 ** -127))
                unit = _power(torch.where(f == 0.5, e - 1, e))
            codes = _nearest(y / torch.where(unit > 0, unit, 1.0)[:, None], 2, 0).clamp(-6.0, 6.0)
            back[a:a + 8192, b:b + block] = codes * unit[:, None]
    return dict(back=back, row_scale=row_scale)


def _power(e):
    """2^e in 64 bits, exactly, from whole exponents."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest(x, digits, least):
    """The nearest number of so many significant bits whose exponent is `least` or more; ties to even."""
    _, e = torch.frexp(x.abs().clamp(min=2.0 ** least))
    step = _power(e - digits)
    return torch.round(x / step) * step


def _exact_head(state):
    case = state["case"]
    k, block, rows, vocab = case["k"], case["block"], case["rows"], case["vocab"]

    def columns(packed, scales, row_scale, b):
        """128 columns of an operand from column b on: 2^(e - 1) (1 + m / 2), or m / 2 where e is 0, by the scales."""
        n = packed.shape[0]
        at = torch.arange(b, min(b + 128, k), device=DEVICE)
        c = (packed[:, at // 2].int() >> (4 * (at % 2))[None]) & 15
        e, m = (c >> 1) & 3, (c & 1).double()
        v = torch.where(e > 0, (1.0 + m / 2) * _power(e - 1), m / 2) * torch.where(c > 7, -1.0, 1.0)
        r, j = torch.arange(n, device=DEVICE)[:, None], (at // block)[None]
        tile = r // 128 * _scale_tiles(n, k, block)[1] + j // 4
        byte = scales[tile * 512 + r % 32 * 16 + r // 32 % 4 * 4 + j % 4].int()
        if block == 16:
            e, m = (byte >> 3) & 15, (byte & 7).double()
            s = torch.where(e > 0, (1.0 + m / 8) * _power(e - 7), m * 2.0 ** -9)
        else:
            s = _power(byte - 127)
        return v * (s if row_scale is None else s * row_scale.double()[:, None])

    out = torch.zeros((rows, vocab), dtype=torch.float64, device=DEVICE)
    for b in range(0, k, 128):
        out.addmm_(columns(state["hidden"], state["hidden_scale"], state["hidden_row_scale"], b),
                   columns(state["weight"], state["weight_scale"], state["weight_row_scale"], b).t())
    return out
