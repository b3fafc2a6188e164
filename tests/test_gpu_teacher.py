"""The most likely tokens of rows and distillation from them, on the GPU against their
definitions in double precision (oracle/teacher.py). Needs a GB300.

Tokens are equal. Tolerances of the other outputs, from the kernels' fp32 arithmetic (EPS =
2^-24, one rounding; depths in nats below the row's largest):
 - an exponential: 2^-22 of itself (ex2.approx; exp2f and expf are within that), and three
   roundings of its argument;
 - a sum of A terms one after another: 4 sqrt(A) EPS of itself (Higham and Mary, lambda = 4),
   A at most V / 256 + 64 in a thread and the joins after it;
 - a row's sum S and the sum outside the list, each of the two; a logprob adds the roundings
   of its own two terms and of the output;
 - a divergence is added up in double from logprobs that share ln S, masses q within 4 EPS;
 - the gradient is p W - q from p and q with these errors (outside the list p_v / p_out times
   W p_out - q_out), and half a step of its type.
"""
import numpy as np
import pytest

import oracle.teacher as O
import workloads

pytestmark = pytest.mark.gpu
EPS, EXP = 2.0 ** -24, 2.0 ** -22
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = 2.0 ** -125  # below it fp32 has fewer digits, and exponentials are 0


@pytest.fixture(scope="module")
def sampler():
    from decode_step_token_gb300 import build
    build.build_library()
    import decode_step_token_gb300 as d
    s = d.Sampler(max_rows=2048, max_vocab=262144)
    yield s
    s.close()


def _round(x, kind):
    if kind == "f32":
        return x.astype(np.float32)
    return workloads.bf16_bits_to_f32(workloads.to_bf16_bits(x.astype(np.float32))).reshape(x.shape)


def _dev(a):
    import torch

    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")


def _buffer(n, V, kind, pad, shift, fill):
    """(whole buffer, its [n, V] part with rows V + pad apart)."""
    import torch

    t = torch.bfloat16 if kind == "bf16" else torch.float32
    flat = torch.full((n * (V + pad) + shift + 64,), fill, dtype=t, device="cuda:0")
    return flat, flat[shift:shift + n * (V + pad)].view(n, V + pad)[:, :V]


def _logits(x, kind, pad=0, shift=0):
    import torch

    flat, view = _buffer(*x.shape, kind, pad, shift, float("nan"))
    view.copy_(torch.from_numpy(x))
    return view


def _depths(logp):
    return np.where(np.isfinite(logp), logp.max() - logp, 0.0)


def _sum_error(p, depth, V):
    """Relative error of the sum of p's exponentials."""
    total = p.sum()
    return EXP + 3 * EPS * ((p * depth).sum() / total if total > 0 else 0) + 4.0 * np.sqrt(V / 256 + 64) * EPS


def _same(a, b, tol, what):
    assert np.array_equal(np.isnan(a), np.isnan(b)), what
    fine = np.isfinite(b)
    assert np.array_equal(a[~fine & ~np.isnan(b)], b[~fine & ~np.isnan(b)]), what
    bad = ~(np.abs(a[fine] - b[fine]) <= np.broadcast_to(tol, b.shape)[fine])
    assert not bad.any(), (what, np.argwhere(fine)[bad][:5], a[fine][bad][:5], b[fine][bad][:5])


# ------------------------------------------------------------------------------- the most likely tokens
def _run_top(sampler, x, kind, n, pad=0, shift=0, tokens=None, T=None, weight=None, entropy=True, stream=None):
    import torch

    rows = x.shape[0]
    out = dict(ids=torch.full((rows, n), -7, dtype=torch.int32, device="cuda:0"),
               logprobs=torch.full((rows, n), -7.0, device="cuda:0"), rest=torch.full((rows,), -7.0, device="cuda:0"),
               status=torch.full((rows,), -7, dtype=torch.int32, device="cuda:0"))
    if tokens is not None:
        out["logprob"] = torch.full((rows,), -7.0, device="cuda:0")
    if entropy:
        out["entropy"] = torch.full((rows,), -7.0, device="cuda:0")
    sampler.score_top(logits=_logits(x, kind, pad, shift), top_n=n, tokens=_dev(tokens), temperature=_dev(T),
                      weight=_dev(weight), out_top_ids=out["ids"], out_top_logprobs=out["logprobs"],
                      out_rest_logprob=out["rest"], out_logprob=out.get("logprob"), out_entropy=out.get("entropy"),
                      out_status=out["status"])
    return {k: v.cpu().numpy() if v.dtype == torch.int32 else v.double().cpu().numpy() for k, v in out.items()}


def _check_top(got, x, n, tokens=None, T=None, weight=None):
    rows, V = x.shape
    want = O.top(x, n, tokens, T, weight)
    np.testing.assert_array_equal(got["status"], want["status"])
    np.testing.assert_array_equal(got["ids"], want["ids"])
    for r in range(rows):
        if want["status"][r] != 0 or (weight is not None and weight[r] == 0):
            for k in ("logprobs", "rest", "logprob", "entropy"):
                if k in got:
                    np.testing.assert_array_equal(got[k][r], want[k][r])
            continue
        y = x[r].astype(np.float64) / (1.0 if T is None or T[r] < np.float32(1e-5) else float(T[r]))
        logp = y - y.max()
        logp = logp - O.log_sum(logp)
        p, depth = np.exp(logp), _depths(logp)
        s = _sum_error(p, depth, V)
        ids = want["ids"][r][want["ids"][r] >= 0]
        m = len(ids)
        _same(got["logprobs"][r, :m], want["logprobs"][r, :m], s + 2 * EPS + 3 * EPS * depth[ids] + EPS * np.abs(logp[ids]), "logprobs")
        assert (got["logprobs"][r, m:] == -np.inf).all()
        outside = np.ones(V, bool)
        outside[ids] = False
        if want["rest"][r] > -80:
            # the exponentials are relative to the list's least, which is within the row
            near = depth[ids].max() if m else 0
            s_out = _sum_error(p[outside], depth[outside], V) + 3 * EPS * near
            _same(got["rest"][r:r + 1], want["rest"][r:r + 1], s + s_out + 4 * EPS + EPS * abs(want["rest"][r]), "rest")
        else:
            assert got["rest"][r] < -79
        if "logprob" in got:
            t = tokens[r]
            _same(got["logprob"][r:r + 1], np.maximum(want["logprob"][r:r + 1], -np.inf),
                  s + 2 * EPS + 3 * EPS * depth[t] + EPS * np.abs(want["logprob"][r]), "logprob")
        if "entropy" in got:
            far = (p * depth).sum() + depth[ids].max()
            tol = s * (1 + far) + far * (EXP + s) + 6 * EPS * ((p * depth ** 2).sum() + far ** 2) + EPS * abs(want["entropy"][r])
            _same(got["entropy"][r:r + 1], want["entropy"][r:r + 1], tol + 2 * EPS, "entropy")


TOPS = [  # rows, vocabulary, n, type, pad, shift, heat, kept, banned, entropy
    (1, 1, 1, "f32", 0, 0, False, 1.0, 0.0, True), (3, 2, 5, "bf16", 0, 1, True, 1.0, 0.0, True),
    (2, 7, 128, "f32", 3, 1, False, 1.0, 0.3, True), (5, 100, 20, "bf16", 5, 3, True, 1.0, 0.0, False),
    (4, 1000, 128, "f32", 0, 0, False, 1.0, 0.0, True), (9, 1023, 1, "bf16", 1, 0, True, 0.6, 0.2, True),
    (70, 2051, 64, "bf16", 0, 5, True, 0.8, 0.0, True), (33, 8191, 100, "f32", 2, 2, True, 0.7, 0.5, True),
    (1, 50257, 128, "bf16", 0, 0, False, 1.0, 0.0, True), (1, 151936, 20, "bf16", 0, 0, True, 1.0, 0.0, False),
    (32, 151936, 20, "bf16", 0, 0, True, 1.0, 0.0, False), (7, 128000, 128, "f32", 1, 1, True, 1.0, 0.1, True),
    (2, 262144, 17, "f32", 0, 0, False, 1.0, 0.0, True), (3, 262143, 128, "bf16", 1, 7, True, 1.0, 0.9, True),
    (310, 9001, 40, "bf16", 0, 0, True, 0.9, 0.0, False), (1500, 700, 64, "f32", 1, 0, False, 0.9, 0.0, True),
    (400, 33000, 64, "bf16", 8, 0, False, 0.5, 0.0, False), (200, 20000, 128, "f32", 0, 0, True, 1.0, 0.999, True)]


@pytest.mark.parametrize("shape", TOPS)
def test_top(sampler, shape):
    rows, V, n, kind, pad, shift, heat, kept, banned, entropy = shape
    rng = np.random.default_rng(rows * 31 + V)
    x = 2.0 * rng.standard_normal((rows, V))
    if banned:
        x[rng.random((rows, V)) < banned] = -np.inf
    tokens = rng.integers(0, V, rows).astype(np.int32)
    x[np.arange(rows), tokens] = rng.uniform(0, 9, rows)
    x = _round(x, kind)
    T = rng.uniform(0.5, 1.6, rows).astype(np.float32) if heat else None
    weight = None
    if kept < 1:
        weight = (rng.random(rows) < kept).astype(np.float32)
        x[weight == 0] = np.nan
    tokens = tokens if rows % 2 else None
    got = _run_top(sampler, x, kind, n, pad, shift, tokens, T, weight, entropy)
    _check_top(got, x, n, tokens, T, weight)


@pytest.mark.parametrize("V", [1, 2, 31, 127, 128, 257, 500, 1025, 4095, 4096, 4103, 8185, 8186, 8192, 8200])
@pytest.mark.parametrize("n", [1, 8, 128])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_top_short_rows(sampler, V, n, kind):
    """Rows that one warp takes, and a little longer ones; they begin anywhere, and some are flat, or nearly so."""
    rng = np.random.default_rng(V + n)
    rows = 1300 if V < 600 else 170
    x = rng.standard_normal((rows, V)) * rng.choice([0.001, 1.0, 30.0], (rows, 1))
    x[rng.random((rows, V)) < 0.02] = -np.inf
    x[3], x[5, V // 2:], x[7] = 0.25, -np.inf, rng.integers(0, 2, V)
    x = _round(x, kind)
    weight = (rng.random(rows) < 0.9).astype(np.float32)
    x[weight == 0] = np.nan
    T = rng.uniform(0.5, 1.6, rows).astype(np.float32)
    tokens = rng.integers(0, V, rows).astype(np.int32)
    got = _run_top(sampler, x, kind, n, 1 + V % 2, V % 5, tokens, T, weight, n != 8)
    some = np.concatenate([np.arange(min(rows, 160)), np.arange(rows - 10, rows)])
    _check_top({k: v[some] for k, v in got.items()}, x[some], n, tokens[some], T[some], weight[some])


@pytest.mark.parametrize("rows", [300, 700])
@pytest.mark.parametrize("V", [4089, 12001, 16376, 16384, 16385, 16400])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_top_rows_of_warps_where_there_are_many(sampler, V, kind, rows):
    rng = np.random.default_rng(V)
    x = rng.standard_normal((rows, V if kind == "bf16" else V // 2))
    x[2], x[4] = np.sort(x[2]), 1.0
    x = _round(x, kind)
    got = _run_top(sampler, x, kind, 64, V % 2, V % 3)
    some = np.concatenate([np.arange(24), np.arange(rows - 8, rows)])
    _check_top({k: v[some] for k, v in got.items()}, x[some], 64)


# parts of rows that leave more keys than are ranked at once
@pytest.mark.parametrize("rows,V,n", [(6, 157971, 18), (17, 60001, 99), (2, 262144, 128), (3, 100000, 12), (60, 50000, 65)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("order", ["random", "one part", "flat", "few"])
def test_top_joined_parts(sampler, rows, V, n, kind, order):
    rng = np.random.default_rng(V + n)
    x = rng.standard_normal((rows, V))
    if order == "one part":  # all that are wanted, and more, are next to each other
        x[:, V // 3:V // 3 + 4 * n] += 20
    elif order == "flat":
        x = rng.integers(0, 2, (rows, V)) * 0.5
    elif order == "few":  # parts with fewer than n
        x = np.where(rng.random((rows, V)) < 300 / V, x, -np.inf)
    x = _round(x, kind)
    _check_top(_run_top(sampler, x, kind, n), x, n)


@pytest.mark.parametrize("V,n", [(300, 128), (9000, 5), (40000, 128), (151936, 64)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [6, 700])
def test_top_orders_and_ties(sampler, V, n, kind, rows):
    """Rows in rising and falling order, flat ones, few different values, zeros of both signs, one finite token."""
    if rows * V > 30_000_000:
        rows = 320
    rng = np.random.default_rng(V)
    x = np.empty((rows, V))
    up = np.sort(3 * rng.standard_normal(V))
    for r in range(rows):
        x[r] = [lambda: up, lambda: up[::-1], lambda: np.full(V, 1.5), lambda: rng.integers(0, 3, V),
                lambda: np.where(rng.random(V) < 0.5, 0.0, -0.0), lambda: np.where(np.arange(V) == V - 2, 1.0, -np.inf)][r % 6]()
    x = _round(x, kind)
    if rows > 6:  # only some of the rows on the host
        some = np.concatenate([np.arange(12), np.arange(rows - 6, rows)])
        got = _run_top(sampler, x, kind, n)
        got = {k: v[some] for k, v in got.items()}
        x = x[some]
    else:
        got = _run_top(sampler, x, kind, n)
    _check_top(got, x, n)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [200, 30000])
def test_top_extreme_values(sampler, kind, V):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((8, V))
    x[0] *= 1e4  # one token has all the mass
    x[1] = 3e38 * np.sign(x[1])
    x[2] = -3e38
    x[3] = np.where(np.arange(V) % 2 == 0, -3.38e38, -np.inf)
    x[4] *= 1e-40 if kind == "f32" else 1e-30
    x[5, 3] = 100.0
    x = _round(x, kind)
    T = np.array([1, 1, 1, 1, 1, 1, 0.02, 50], np.float32)
    got = _run_top(sampler, x, kind, 16, T=T, entropy=False)
    _check_top(got, x, 16, T=T)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", [(9, 5000), (9, 100000), (640, 5000)])
def test_top_status_rows(sampler, kind, rows, V):
    rng = np.random.default_rng(6)
    x = rng.standard_normal((rows, V))
    T, tokens = np.ones(rows, np.float32), rng.integers(0, V, rows).astype(np.int32)
    x[0, V // 2], x[1, 0], x[2] = np.nan, np.inf, -np.inf
    T[3], T[4], T[5] = -1, np.nan, np.inf
    tokens[6], tokens[7] = -1, V
    T[8] = 1e-6  # greedy: T = 1
    x = _round(x, kind)
    _check_top(_run_top(sampler, x, kind, 8, tokens=tokens, T=T), x, 8, tokens, T)


# ------------------------------------------------------------------------------- distillation
class Batch:
    def __init__(self, seed, rows, V, k, kind="f32", pad=0, shift=0, heat=False, kept=1.0, tail=True, coef=0.0, short=0.0,
                 scale=2.0, noise=0.7):
        rng = self.rng = np.random.default_rng(seed)
        self.kind, self.pad, self.shift, self.coef, self.k = kind, pad, shift, coef, k
        x = scale * rng.standard_normal((rows, V))
        self.tokens = rng.integers(0, V, rows).astype(np.int32)
        x[np.arange(rows), self.tokens] = rng.uniform(0, 9, rows)
        self.x = _round(x, kind)
        self.T = rng.uniform(0.5, 1.6, rows).astype(np.float32) if heat else None
        z = (self.x + noise * rng.standard_normal((rows, V))) / (1.0 if self.T is None else self.T[:, None])
        lp = z - z.max(1, keepdims=True)
        lp -= np.log(np.exp(lp).sum(1, keepdims=True))
        m = min(k, V)
        best = np.argsort(-lp, 1, kind="stable")[:, :m]
        self.ids, self.l = np.full((rows, k), -1, np.int32), np.full((rows, k), -np.inf, np.float32)
        count = np.where(rng.random(rows) < short, rng.integers(0, m + 1, rows), m)
        self.rest = np.empty(rows, np.float32)
        for r in range(rows):
            at = best[r, :count[r]]
            self.ids[r, :count[r]], self.l[r, :count[r]] = at, lp[r, at]
            self.rest[r] = O.log_sum(np.delete(lp[r], at))
        if not tail:
            self.rest = None
        self.weight = rng.uniform(0.2, 1.0, rows).astype(np.float32)
        if kept < 1:
            self.weight[rng.random(rows) >= kept] = 0
            self.x[self.weight == 0] = np.nan

    def run(self, sampler, grad=True, in_place=False, scale=1.5, scale_dev=None, out=None):
        import torch

        rows, V = self.x.shape
        self.logits = _logits(self.x, self.kind, self.pad, self.shift)
        self.gflat = None
        if grad:
            self.gflat, g = _buffer(rows, V, self.kind, self.pad, self.shift, -7.0)
            if in_place:
                g = self.logits
        else:
            g = None
        self.scale = scale * (1.0 if scale_dev is None else scale_dev)
        o = dict(loss=torch.full((1,), -7.0, device="cuda:0"), kl=torch.full((rows,), -7.0, device="cuda:0"),
                 logprob=torch.full((rows,), -7.0, device="cuda:0"),
                 status=torch.full((rows,), -7, dtype=torch.int32, device="cuda:0"))
        self.call = lambda: sampler.distill_loss(
            logits=self.logits, teacher_ids=self.d[0], teacher_logprobs=self.d[1], teacher_rest=self.d[2], tokens=self.d[3],
            token_coef=self.coef, temperature=self.d[4], weight=self.d[5], grad_scale=scale, grad_scale_dev=self.d[6],
            out_loss=o["loss"], out_kl=o["kl"], out_logprob=o["logprob"], out_status=o["status"], out_grad=g)
        self.d = [_dev(a) for a in (self.ids, self.l, self.rest, self.tokens, self.T, self.weight,
                                    None if scale_dev is None else np.array([scale_dev], np.float32))]
        self.call()
        self.out, self.grad = o, g
        return self

    def check(self):
        import torch

        rows, V = self.x.shape
        want = O.distill(self.x, self.ids, self.l, self.rest, self.tokens, self.coef, self.T, self.weight, self.scale)
        got = {k: v.cpu().numpy() if v.dtype == torch.int32 else v.double().cpu().numpy() for k, v in self.out.items()}
        np.testing.assert_array_equal(got["status"], want["status"])
        g = None if self.grad is None else self.grad.double().cpu().numpy()
        loss_tol = EPS * abs(want["loss"])
        for r in range(rows):
            w = float(self.weight[r])
            if w == 0 or want["status"][r]:
                for k in ("kl", "logprob"):
                    np.testing.assert_array_equal(got[k][r], want[k][r])
                if g is not None:
                    np.testing.assert_array_equal(g[r], want["grad"][r])
                continue
            T = 1.0 if self.T is None or self.T[r] < np.float32(1e-5) else float(self.T[r])
            y = self.x[r].astype(np.float64) / T
            logp = y - y.max()
            logp = logp - O.log_sum(logp)
            p, depth = np.exp(logp), _depths(logp)
            s = _sum_error(p, depth, V) + 2 * EPS
            ids, l = self.ids[r][self.ids[r] >= 0], self.l[r][self.ids[r] >= 0].astype(np.float64)
            q, tail = np.exp(l), -np.inf if self.rest is None else float(self.rest[r])
            qr = np.exp(tail)
            outside = np.ones(V, bool)
            outside[ids] = False
            s_out, ln_out, top_out = 0.0, -np.inf, 0.0
            if p[outside].sum() > 0:
                s_out = _sum_error(p[outside], depth[outside], V) + 2 * EPS
                ln_out, top_out = O.log_sum(logp[outside]), depth[outside][np.isfinite(logp[outside])].min()
            total = q.sum() + qr + self.coef
            with np.errstate(invalid="ignore"):
                terms = np.where(q > 0, q * np.abs(l - logp[ids]), 0.0)
                tol = (q.sum() + qr) * s + 6 * EPS * terms.sum() + EPS * abs(want["kl"][r])
                if qr > 0:
                    tol += qr * (s_out + 6 * EPS * abs(tail - ln_out))
            _same(got["kl"][r:r + 1], want["kl"][r:r + 1], tol, "kl")
            t = self.tokens[r]
            tol_lp = s + 2 * EPS + 3 * EPS * depth[t] + EPS * abs(want["logprob"][r])
            _same(got["logprob"][r:r + 1], want["logprob"][r:r + 1], tol_lp, "logprob")
            loss_tol += w * (tol + self.coef * tol_lp)
            if g is None:
                continue
            gw = w * abs(self.scale) / T
            err = np.empty(V)
            each = EXP + s + s_out + 3 * EPS * (depth + 2 * top_out) + 16 * EPS
            err = (total * p + (qr * np.exp(logp - ln_out) if ln_out > -np.inf else 0.0)) * each
            err[ids] = total * p[ids] * (EXP + s + 3 * EPS * depth[ids] + 16 * EPS) + q * 16 * EPS
            err[t] += self.coef * 16 * EPS
            tol = gw * err * 1.01 + HALF[self.kind] * np.abs(want["grad"][r]) * 1.01 + TINY
            bad = ~(np.abs(g[r] - want["grad"][r]) <= tol)
            assert not bad.any(), (r, np.nonzero(bad)[0][:5], g[r][bad][:5], want["grad"][r][bad][:5], tol[bad][:5])
        _same(got["loss"], np.array([want["loss"]]), loss_tol, "loss")
        if self.gflat is not None and self.grad.data_ptr() != self.logits.data_ptr():
            beside = torch.ones_like(self.gflat, dtype=torch.bool)
            beside[self.shift:self.shift + rows * (V + self.pad)].view(rows, -1)[:, :V] = False
            assert bool((self.gflat[beside] == -7.0).all()), "written beside the gradient"


DISTILS = [  # rows, vocabulary, list, type, pad, shift, heat, kept, tail, coef, short
    (1, 1, 1, "f32", 0, 0, False, 1.0, True, 0.0, 0.0), (3, 2, 5, "bf16", 0, 1, True, 1.0, True, 0.5, 0.5),
    (2, 7, 128, "f32", 3, 1, False, 1.0, True, 0.0, 0.0), (5, 100, 20, "bf16", 5, 3, True, 1.0, False, 0.2, 0.0),
    (4, 1024, 8, "f32", 0, 0, False, 1.0, True, 0.0, 0.0), (9, 1023, 1, "bf16", 1, 0, True, 0.6, True, 0.0, 0.0),
    (70, 2051, 64, "bf16", 0, 5, True, 0.8, True, 0.1, 0.3), (33, 8191, 100, "f32", 2, 2, True, 0.7, False, 0.3, 0.5),
    (1, 50257, 128, "bf16", 0, 0, False, 1.0, True, 0.0, 0.0), (1, 151936, 20, "bf16", 0, 0, True, 1.0, True, 1.0, 0.0),
    (12, 151936, 64, "bf16", 8, 0, True, 1.0, True, 0.0, 0.0), (7, 128000, 100, "f32", 1, 1, True, 1.0, True, 0.1, 0.5),
    (2, 262144, 17, "f32", 0, 0, False, 1.0, True, 0.0, 0.0), (3, 262143, 128, "bf16", 1, 7, True, 1.0, True, 0.2, 0.0),
    (2, 262143, 64, "f32", 3, 2, True, 1.0, False, 0.2, 0.0), (310, 9001, 40, "bf16", 0, 0, True, 0.9, True, 0.0, 0.0),
    (1500, 700, 64, "f32", 1, 0, False, 0.9, True, 0.3, 0.2), (400, 33000, 64, "bf16", 8, 0, False, 0.5, True, 0.1, 0.0),
    (500, 20011, 128, "f32", 0, 0, True, 1.0, True, 0.0, 0.0)]


@pytest.mark.parametrize("rows,V,kind", [(140, 80000, "f32"), (60, 151936, "bf16"), (100, 40961, "f32"), (50, 230001, "bf16"),
                                         (90, 151936, "f32"), (40, 262144, "f32"), (500, 16385, "bf16"), (700, 8191, "f32")])
def test_distill_on_clusters_of_all_sizes(sampler, rows, V, kind):
    """More rows than there are clusters, of sizes that are no powers of two among them; the same bits again."""
    import torch

    b = Batch(V, rows, V, 33, kind, pad=V % 2, heat=True, coef=0.1, kept=0.9)
    b.run(sampler).check()
    grad, kl = b.grad.clone(), b.out["kl"].clone()
    for _ in range(3):
        b.call()
    assert torch.equal(torch.nan_to_num(b.grad.float()), torch.nan_to_num(grad.float())) and torch.equal(b.out["kl"], kl)


@pytest.mark.parametrize("shape", DISTILS)
@pytest.mark.parametrize("grad", [True, False])
def test_distill(sampler, shape, grad):
    rows, V, k, kind, pad, shift, heat, kept, tail, coef, short = shape
    b = Batch(rows * 37 + V, rows, V, k, kind, pad, shift, heat, kept, tail, coef, short)
    b.run(sampler, grad=grad).check()


@pytest.mark.parametrize("V,kind", [(5003, "bf16"), (151937, "bf16"), (128000, "f32"), (300, "f32")])
def test_distill_in_place_with_a_scale_on_the_device(sampler, V, kind):
    Batch(V, 9, V, 30, kind, pad=1, heat=True, coef=0.2, kept=0.8).run(sampler, in_place=True, scale_dev=0.75).check()


def test_gradient_against_differences(sampler):
    """The loss itself, as the kernel computes it, moved along the gradient."""
    b = Batch(3, 6, 900, 12, heat=True, coef=0.3)
    b.run(sampler, scale=1.0)
    g = b.grad.double().cpu().numpy()
    d = b.rng.standard_normal(b.x.shape)
    x, h = b.x.copy(), 0.05
    vals = []
    for sign in (1, -1):
        b.x = (x + sign * h * d).astype(np.float32)
        vals.append(b.run(sampler, grad=False, scale=1.0).out["loss"].item())
    # third derivatives of a log-sum are below 1 along d's few units; the loss has 2^-24 of itself
    np.testing.assert_allclose((g * d).sum(), (vals[0] - vals[1]) / (2 * h), rtol=2e-2, atol=2e-3)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [3000, 130000])
def test_distill_status_rows(sampler, kind, V):
    b = Batch(V, 16, V, 10, kind, coef=0.2)
    b.T = np.ones(16, np.float32)
    b.x[0, V // 2], b.x[1, b.ids[1, 4]], b.x[2, 0], b.x[3] = np.nan, np.inf, np.inf, -np.inf
    b.T[4], b.T[5], b.T[6] = -1, np.nan, 1e-6
    b.tokens[7], b.tokens[8] = -1, V
    b.ids[9, 3], b.ids[10, 2], b.ids[11, 7] = V, -2, b.ids[11, 1]  # outside, outside, twice
    b.l[12, 4], b.l[13, 0], b.rest[14] = np.nan, np.inf, np.nan
    b.ids[15] = -1  # an empty list
    b.run(sampler).check()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [400, 60000])
def test_distill_without_mass(sampler, kind, V):
    """Tokens of the list, and all tokens outside it, that the student forbids; masses that are far apart."""
    b = Batch(V, 6, V, 10, kind)
    b.x[0, b.ids[0, 3]] = -np.inf  # an infinite divergence, with a finite gradient
    outside = np.ones(V, bool)
    outside[b.ids[1]] = False
    b.x[1, outside] = -np.inf
    b.l[2, 5] = -np.inf            # a token of no mass in the teacher
    b.x[2, b.ids[2, 5]] = -np.inf
    b.x[3, b.ids[3]] = 60.0        # nothing is left outside, but for the logarithm
    b.rest[4] = -np.inf
    b.x[5, b.ids[5]] = -60.0
    b.run(sampler).check()


def test_teacher_to_student(sampler):
    """The lists of score_top into distill_loss: the teacher's own rows have no divergence and no gradient."""
    import torch

    for kind in ("bf16", "f32"):
        rng = np.random.default_rng(8)
        x = _round(2 * rng.standard_normal((40, 30011)), kind)
        T = rng.uniform(0.5, 1.5, 40).astype(np.float32)
        logits = _logits(x, kind)
        ids = torch.empty((40, 64), dtype=torch.int32, device="cuda:0")
        lps, rest, kl = torch.empty((40, 64), device="cuda:0"), torch.empty(40, device="cuda:0"), torch.empty(40, device="cuda:0")
        loss, grad = torch.empty(1, device="cuda:0"), torch.empty_like(logits)
        sampler.score_top(logits=logits, top_n=64, temperature=_dev(T), out_top_ids=ids, out_top_logprobs=lps,
                          out_rest_logprob=rest)
        sampler.distill_loss(logits=logits, temperature=_dev(T), teacher_ids=ids, teacher_logprobs=lps, teacher_rest=rest,
                             out_loss=loss, out_kl=kl, out_grad=grad)
        # both have errors of a sum of 30011 exponentials, and logprobs of up to 15 in fp32
        assert kl.abs().max().item() < 2 * (EXP + 4 * np.sqrt(30011 / 256 + 64) * EPS + 3 * EPS * 15 + 16 * EPS)
        lp = torch.log_softmax(logits.double() / _dev(T).double()[:, None], 1).exp()
        assert (grad.double().abs() * _dev(T).double()[:, None] <= lp * 1e-5 + 1e-30).all()


@pytest.mark.parametrize("rows,V", [(3, 151936), (50, 3000), (700, 9001)])
def test_same_bits_each_time_and_in_a_graph(sampler, rows, V):
    """Also on another stream, and while an eager call's outputs live on."""
    import torch

    b = Batch(rows, rows, V, 50, "bf16", heat=True, coef=0.1, kept=0.9)
    b.run(sampler)
    top = [torch.empty((rows, 50), dtype=torch.int32, device="cuda:0"), torch.empty((rows, 50), device="cuda:0"),
           torch.empty(rows, device="cuda:0"), torch.empty(rows, device="cuda:0")]

    def both():
        sampler.score_top(logits=b.logits, top_n=50, temperature=b.d[4], weight=b.d[5], out_top_ids=top[0],
                          out_top_logprobs=top[1], out_rest_logprob=top[2], out_entropy=top[3])
        b.call()

    both()
    outs = top + [b.out["loss"], b.out["kl"], b.grad]
    first = [t.clone() for t in outs]

    def same():
        torch.cuda.synchronize()
        for t, f in zip(outs, first):
            assert torch.equal(t.view(torch.uint8), f.view(torch.uint8))
            t.zero_()

    same()
    for _ in range(3):
        both()
        same()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        both()
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(3):
        graph.replay()
        same()


def test_nothing_to_do(sampler):
    import torch

    x, f = torch.empty((0, 50), device="cuda:0"), torch.empty(0, device="cuda:0")
    ids, lps = torch.empty((0, 4), dtype=torch.int32, device="cuda:0"), torch.empty((0, 4), device="cuda:0")
    loss = torch.full((1,), -7.0, device="cuda:0")
    sampler.score_top(logits=x, top_n=4, out_top_ids=ids, out_top_logprobs=lps)
    sampler.distill_loss(logits=x, teacher_ids=ids, teacher_logprobs=lps, out_loss=loss, out_kl=f)
    assert loss.item() == 0
    # rows that are all left out
    x = torch.full((5, 50), float("nan"), device="cuda:0")
    ids, lps = torch.zeros((5, 4), dtype=torch.int32, device="cuda:0"), torch.zeros((5, 4), device="cuda:0")
    w, grad = torch.zeros(5, device="cuda:0"), torch.full((5, 50), -7.0, device="cuda:0")
    sampler.distill_loss(logits=x, teacher_ids=ids, teacher_logprobs=lps, weight=w, out_loss=loss, out_grad=grad)
    assert loss.item() == 0 and (grad == 0).all()
    sampler.score_top(logits=x, top_n=4, weight=w, out_top_ids=ids, out_top_logprobs=lps)
    assert (ids == -1).all() and (lps == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", [(3, 3000), (3, 151936), (400, 3000)])
def test_waits_that_give_up(kind, rows, V):
    import decode_step_token_gb300 as d

    b = Batch(1, rows, V, 20, kind, kept=0.8)
    with d.Sampler(max_rows=512, max_vocab=262144, short_waits=True) as s:
        b.run(s)
        live = b.weight != 0
        assert (b.out["status"].cpu().numpy() == np.where(live, 5, 0)).all()
        kl, g = b.out["kl"].cpu().numpy(), b.grad.float().cpu().numpy()
        assert np.isnan(kl[live]).all() and (kl[~live] == 0).all() and np.isnan(b.out["loss"].item())
        assert np.isnan(g[live]).all() and (g[~live] == 0).all()
        got = _run_top(s, b.x, kind, 9, weight=b.weight)
        assert (got["status"] == np.where(live, 5, 0)).all() and (got["ids"] == -1).all()
        assert np.isnan(got["logprobs"][live]).all() and (got["logprobs"][~live] == 0).all()
    with d.Sampler(max_rows=512, max_vocab=262144) as s:  # nothing is left over
        if rows <= 3:
            b.run(s).check()
            _check_top(_run_top(s, b.x, kind, 9, weight=b.weight), b.x, 9, weight=b.weight)


def test_two_graphs_share_a_workspace(sampler):
    """Graphs of both operators on one handle, of rows in parts and whole ones, replayed in turn on inputs that change."""
    import torch

    gen = torch.Generator(device="cuda:0").manual_seed(11)
    sets = []
    for rows, V in ((3, 151936), (40, 100000), (400, 5000)):
        x = torch.randn((rows, V), generator=gen, device="cuda:0")
        o = dict(ids=torch.empty((rows, 20), dtype=torch.int32, device="cuda:0"), lps=torch.empty((rows, 20), device="cuda:0"),
                 rest=torch.empty(rows, device="cuda:0"), loss=torch.empty(1, device="cuda:0"), grad=torch.empty_like(x))

        def call(x=x, o=o):
            sampler.score_top(logits=x, top_n=20, out_top_ids=o["ids"], out_top_logprobs=o["lps"], out_rest_logprob=o["rest"])
            sampler.distill_loss(logits=0.7 * x, teacher_ids=o["ids"], teacher_logprobs=o["lps"], teacher_rest=o["rest"],
                                 out_loss=o["loss"], out_grad=o["grad"])

        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        sets.append((x, o, call, graph))
    for turn in range(4):
        for x, o, call, graph in sets:
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda:0"))
        for x, o, call, graph in sets:
            graph.replay()
        torch.cuda.synchronize()
        for x, o, call, graph in sets:
            first = {k: v.clone() for k, v in o.items()}
            call()
            torch.cuda.synchronize()
            assert all(torch.equal(first[k], o[k]) for k in o)


@pytest.mark.parametrize("V", [700, 40000, 200001])
def test_rows_far_apart(sampler, V):
    """Offsets beyond 32 bits, of the logits and of the gradient, give what rows side by side give."""
    import torch

    rows, stride = 5, 600_000_001
    gen = torch.Generator(device="cuda:0").manual_seed(V)
    near = torch.randn((rows, V), generator=gen, device="cuda:0").to(torch.bfloat16)
    far = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda:0").view(rows, stride)[:, :V]
    far.copy_(near)
    outs = []
    for x in (near, far):
        ids = torch.empty((rows, 30), dtype=torch.int32, device="cuda:0")
        lps, rest = torch.empty((rows, 30), device="cuda:0"), torch.empty(rows, device="cuda:0")
        sampler.score_top(logits=x, top_n=30, out_top_ids=ids, out_top_logprobs=lps, out_rest_logprob=rest)
        outs.append((ids, lps, rest))
    assert torch.equal(outs[0][0], outs[1][0])
    # rows that begin elsewhere in a vector add up in another order: 4 sqrt(V / 256 + 64) roundings of 2^-24 for each
    for a, b in zip(outs[0][1:], outs[1][1:]):
        assert torch.allclose(a, b, rtol=0, atol=1e-5)
    ids, lps, rest = outs[0]
    loss, grads = [], []
    wide = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda:0").view(rows, stride)[:, :V]
    for x, g in ((near, torch.empty_like(near)), (far, wide)):
        out = torch.empty(1, device="cuda:0")
        sampler.distill_loss(logits=x, teacher_ids=ids, teacher_logprobs=lps + 0.1, teacher_rest=rest,
                             out_loss=out, out_grad=g)
        loss.append(out.item())
        grads.append(g.float())
    assert abs(loss[0] - loss[1]) <= 1e-5 * abs(loss[0])
    # a bf16 rounding where the fp32 values differ in their last places
    assert ((grads[0] - grads[1]).abs() <= 2.0 ** -7 * grads[0].abs() + 1e-12).all()


def test_argument_checks(sampler):
    import torch

    x = torch.randn((4, 50), device="cuda:0")
    ids, lps = torch.zeros((4, 3), dtype=torch.int32, device="cuda:0"), torch.zeros((4, 3), device="cuda:0")
    loss = torch.empty(1, device="cuda:0")
    import decode_step_token_gb300 as d
    top = dict(logits=x, top_n=3, out_top_ids=ids, out_top_logprobs=lps)
    for change, error in [(dict(top_n=4), ValueError), (dict(top_n=0), d.SamplerError), (dict(out_top_ids=lps), TypeError),
                          (dict(out_rest_logprob=loss), ValueError), (dict(out_logprob=lps[:, 0].contiguous()), d.SamplerError),
                          (dict(logits=x.half()), TypeError), (dict(vocab=51), ValueError)]:
        with pytest.raises(error):
            sampler.score_top(**{**top, **change})
    dis = dict(logits=x, teacher_ids=ids, teacher_logprobs=lps, out_loss=loss)
    for change, error in [(dict(teacher_ids=ids[:3]), ValueError), (dict(teacher_logprobs=lps[:, :2]), ValueError),
                          (dict(token_coef=0.5), d.SamplerError), (dict(token_coef=-1.0), d.SamplerError),
                          (dict(teacher_rest=lps), None), (dict(teacher_rest=loss), ValueError),
                          (dict(out_grad=x.bfloat16()), TypeError), (dict(out_grad=x[:3]), ValueError),
                          (dict(teacher_ids=ids.t(), teacher_logprobs=lps.t()), ValueError)]:
        if error is None:
            continue
        with pytest.raises(error):
            sampler.distill_loss(**{**dis, **change})


def _lists_under_way(rng, rows, V, chunk, first, kind):
    """Rows whose list is cut while more keys come than a list of 512 holds with those of the next chunk: in chunk
    `first` `second` values above all before, in the next `third` above those, and all of the one after above them."""
    x = 0.01 * rng.standard_normal((rows, V))
    for r in range(rows):
        lanes, deep = rng.integers(1, 129), rng.integers(1, 6)  # of the first chunk, values that pass the first bar
        x[r, rng.permutation(chunk)[:lanes * deep]] = 5 + 1e-4 * rng.random(lanes * deep)
        second, third, at = rng.integers(40, 250), rng.integers(200, 257), first * chunk
        x[r, at + rng.permutation(chunk)[:second]] = 6 + rng.random(second)
        x[r, at + chunk + rng.permutation(chunk)[:third]] = 8 + rng.random(third)
        x[r, at + 2 * chunk:at + 3 * chunk] = 10 + rng.random(chunk)
        if r % 3 == 1:  # the last chunk in steps of its own
            x[r, at + 2 * chunk:at + 3 * chunk] += 0.001 * np.arange(chunk)
    return _round(x, kind)


@pytest.mark.parametrize("n", [1, 8, 20, 64, 100, 128])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_top_chunk_over_a_list_that_a_cut_comes_back_to(sampler, kind, n):
    """Several rows for each CTA, in either pair of its lists."""
    rng = np.random.default_rng(n)
    chunk = 8192 if kind == "bf16" else 4096
    rows, V, kinds = 640, 9 * chunk, 40
    x = np.concatenate([_lists_under_way(rng, kinds // 2, V, chunk, first, kind) for first in (5, 6)])
    x = x[np.arange(rows) * 7 % kinds]
    got = _run_top(sampler, x, kind, n, entropy=n in (8, 64))
    for r in range(kinds, rows):  # the same rows have the same outputs, wherever they are
        for k in got:
            np.testing.assert_array_equal(got[k][r], got[k][r % kinds])
    _check_top({k: v[:kinds] for k, v in got.items()}, x[:kinds], n)


@pytest.mark.parametrize("n", [4, 20, 64])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_top_chunk_over_such_a_list_in_a_part(sampler, kind, n):
    """The same in one of a row's eight parts."""
    rng = np.random.default_rng(n)
    V = 262144
    chunk = 8192 if kind == "bf16" else 4096
    part = V // 8
    x = 0.01 * rng.standard_normal((6, V))
    if part >= 8 * chunk:
        for r in range(6):
            x[r, r * part:(r + 1) * part] = _lists_under_way(rng, 1, part, chunk, 5, kind)[0]
    else:  # parts of four chunks, which are all looked at for the first bar
        for r in range(6):
            x[r, r * part + 3 * chunk:r * part + 4 * chunk] = 10 + rng.random(chunk)
    x = _round(x, kind)
    _check_top(_run_top(sampler, x, kind, n), x, n)


def _check_rest(got, x, n, T=None):
    """The logprob of what is outside the lists, -inf exactly where that has no finite logit, else within the roundings of
    its own sum (a warp's, of V / 32 in a lane, or of the row), of the row's, and of the distances between their largest."""
    rows, V = x.shape
    far = 0
    for r in range(rows):
        logp = x[r].astype(np.float64) / (1.0 if T is None or T[r] < np.float32(1e-5) else float(T[r]))
        logp = logp - logp.max()
        logp -= O.log_sum(logp)
        ids = got["ids"][r][got["ids"][r] >= 0]
        np.testing.assert_array_equal(ids, np.lexsort((np.arange(V), -x[r]))[:min(n, np.isfinite(logp).sum())])
        out = np.delete(logp, ids)
        if not np.isfinite(out).any():
            assert got["rest"][r] == -np.inf, (r, got["rest"][r])
            continue
        want, depth = O.log_sum(out), _depths(out)
        if want < -3.4028236e38:  # below fp32's range
            assert got["rest"][r] == -np.inf, (r, got["rest"][r])
            continue
        gap = min(logp[ids].min() - out.max(), 60.0)  # a sum relative to the list's least: 84 powers of two below it at most
        far += logp[ids].min() - out.max() > 60
        tol = (_sum_error(np.exp(logp), _depths(logp), V) + _sum_error(np.exp(out - out.max()), depth, 8 * V) + 3 * EPS * gap
               + 4 * EPS + EPS * abs(want))
        assert abs(got["rest"][r] - want) <= tol, (r, got["rest"][r], want, tol)
    return far


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", [(40, 200), (40, 4096), (40, 8000), (700, 16000), (40, 30011), (6, 151936), (170, 40000)])
def test_top_rest_far_below_the_list(sampler, kind, rows, V):
    """The mass of the others, however little it is: low temperatures, leads of some logits, tokens forbidden by a large
    negative number or the type's lowest in place of -inf, all others at -inf, as many tokens as were asked for."""
    rng = np.random.default_rng(V)
    for n in (1, 20, 64):
        x = rng.standard_normal((rows, V))
        T = np.ones(rows, np.float32)
        for r in range(rows):
            some = rng.permutation(V)[:n + r % 2]  # n, or one more
            if r % 7 == 0:
                T[r] = rng.choice([0.02, 0.05, 0.1])
                x[r, some] += 12
            elif r % 7 == 1:
                keep = x[r, some]
                x[r] = -1e4 + x[r]
                x[r, some] = keep
            elif r % 7 == 2:
                keep = x[r, some]
                x[r] = -3.38e38
                x[r, some] = keep
            elif r % 7 == 3:
                keep = x[r, some]
                x[r] = -np.inf
                x[r, some] = keep
            elif r % 7 == 4:  # the list's own next keys are far below it, and the rest far below those
                x[r] = -1500 - 500 * rng.random(V)
                x[r, some] = 3 + 0.1 * rng.random(len(some))
                x[r, rng.permutation(V)[:30]] = -700 - 100 * rng.random(30)
            elif r % 7 == 5:  # all that is wanted in one place, and what comes next in another
                x[r] = -300 + x[r]
                x[r, V // 2:V // 2 + n] = 5
                x[r, :3] = -200
        x = _round(x, kind)
        got = _run_top(sampler, x, kind, n, V % 3, V % 5, T=T, entropy=False)
        some = np.arange(rows) if rows < 100 else np.concatenate([np.arange(28), np.arange(rows - 28, rows)])
        far = _check_rest({k: v[some] for k, v in got.items()}, x[some], n, T[some])
        assert far > len(some) // 4


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V,n", [(1, 1), (2, 1), (5, 5), (64, 64), (128, 128), (100, 128), (129, 128)])
def test_top_rest_of_short_vocabularies(sampler, kind, V, n):
    """All tokens listed, or all but one, which may be far below."""
    rng = np.random.default_rng(V)
    x = rng.standard_normal((60, V))
    x[np.arange(60), rng.integers(0, V, 60)] -= rng.choice([0, 100, 1e4, 1e30], 60)
    x = _round(x, kind)
    got = _run_top(sampler, x, kind, n, V % 3, V % 5, entropy=False)
    _check_rest(got, x, n)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V,n", [(4000, 1), (4000, 64), (40000, 1), (40000, 64)])
def test_top_errors_do_not_go_one_way(sampler, kind, V, n):
    """The mean error of many logprobs at a temperature whose log2(e) / T, as the product of two rounded numbers, is off by
    1.9 EPS. All exponents take the float that is nearest to it, so that the error in all of them is of rel * depth, with
    rel that float's own (0.1 EPS here); ex2.approx and the logarithm are off by 1.5e-8 and 3e-8 the same way at most. What
    is left is at random: the output's rounding (uniform, of EPS |logprob|) and the sums' own, by four standard errors."""
    import torch

    rows, T = 2048, np.float32(1.4400320053)
    exact = np.log2(np.e) / float(T)
    rel = abs(float(np.float32(exact)) / exact - 1)
    assert abs(float(np.float32(np.log2(np.e)) * (np.float32(1) / T)) / exact - 1) > 1.5 * EPS and rel < 0.2 * EPS
    gen = torch.Generator(device="cuda:0").manual_seed(V)
    x = 0.5 * torch.randn((rows, V), generator=gen, device="cuda:0")
    x[:, V // 2] = 8 * float(T)  # far above all others, which have most of the mass
    x = x.to(torch.bfloat16) if kind == "bf16" else x
    tokens = torch.randint(0, V, (rows,), generator=gen, device="cuda:0", dtype=torch.int32)
    ids = torch.empty((rows, n), dtype=torch.int32, device="cuda:0")
    lps, lp, rest = torch.empty((rows, n), device="cuda:0"), torch.empty(rows, device="cuda:0"), torch.empty(rows, device="cuda:0")
    sampler.score_top(logits=x, top_n=n, out_top_ids=ids, out_top_logprobs=lps, out_rest_logprob=rest, tokens=tokens,
                      out_logprob=lp, temperature=torch.full((rows,), float(T), device="cuda:0"))
    z = torch.log_softmax(x.double() / float(T), 1)
    depth = (z.exp() * (z.amax(1, keepdim=True) - z)).sum(1).mean().item()
    one_way = rel * depth + 1.5e-8 + 3e-8
    at_random = 4 / rows ** 0.5 * (EXP + 4 * np.sqrt(V / 32 + 64) * EPS / 32 ** 0.5)
    for got, want in ((lp, z.gather(1, tokens.long()[:, None])[:, 0]), (lps[:, -1], z.gather(1, ids[:, -1:].long())[:, 0]),
                      (rest, torch.logsumexp(z.scatter(1, ids.long(), -torch.inf), 1))):
        mean = (got.double() - want).mean().item()
        size = want.abs().mean().item() if got is lp else 0.0
        # (the outputs other than the drawn tokens' are close together: their roundings may go one way)
        step = 0.0 if got is lp else EPS * want.abs().max().item()
        tol = one_way + step + at_random + 4 / rows ** 0.5 * EPS * size / 3 ** 0.5
        assert abs(mean) <= tol, (mean, tol)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [4000, 40000])
def test_distill_errors_do_not_go_one_way(sampler, kind, V):
    """As above, of divergences, logprobs and (fp32) the gradient outside the lists, W p_v: the mean of its errors relative to
    itself. A gradient's exponential has its own mean error, 5e-8 at most."""
    import torch

    rows, T, k = 1024, float(np.float32(1.4400320053)), 4
    exact = np.log2(np.e) / T
    rel = abs(float(np.float32(exact)) / exact - 1)
    gen = torch.Generator(device="cuda:0").manual_seed(V)
    x = 0.5 * torch.randn((rows, V), generator=gen, device="cuda:0")
    x[:, -2] = 8 * T  # comes last, and is outside the lists
    x = x.to(torch.bfloat16) if kind == "bf16" else x
    ids = torch.rand((rows, V - 2), generator=gen, device="cuda:0").argsort(1)[:, :k].to(torch.int32)
    tokens = torch.randint(0, V, (rows,), generator=gen, device="cuda:0", dtype=torch.int32)
    l = torch.log(torch.rand((rows, k), generator=gen, device="cuda:0") / k)
    kl, lp, loss = torch.empty(rows, device="cuda:0"), torch.empty(rows, device="cuda:0"), torch.empty(1, device="cuda:0")
    grad = torch.empty_like(x)
    sampler.distill_loss(logits=x, teacher_ids=ids, teacher_logprobs=l, tokens=tokens, out_loss=loss, out_kl=kl, out_logprob=lp,
                         temperature=torch.full((rows,), T, device="cuda:0"), out_grad=grad)
    z = torch.log_softmax(x.double() / T, 1)
    q = torch.exp(l.double())
    depth = (z.exp() * (z.amax(1, keepdim=True) - z)).sum(1).mean().item()
    one_way = rel * depth + 1.5e-8 + 3e-8
    at_random = 4 / rows ** 0.5 * (EXP + 4 * np.sqrt(V / 256 + 64) * EPS / 32 ** 0.5)
    for got, want in ((lp, z.gather(1, tokens.long()[:, None])[:, 0]), (kl, (q * (l.double() - z.gather(1, ids.long()))).sum(1))):
        mean, size = (got.double() - want).mean().item(), want.abs().mean().item()
        tol = one_way * q.sum(1).max().item() + at_random + 4 / rows ** 0.5 * EPS * (size + 4) / 3 ** 0.5
        assert abs(mean) <= tol, (mean, tol)
    if kind == "f32":
        want = z.exp() * q.sum(1, keepdim=True) / T
        off = (grad.double() - want) / want
        off.scatter_(1, ids.long(), 0.0)
        # (the largest, alone of its kind, is not among them; an element's own roundings are at random)
        mean, far = off[:, :-2].mean().item(), (z[:, -2:-1] - z[:, :-2]).mean().item()
        tol = rel * far + one_way + 5e-8 + 4 * EPS + at_random
        assert abs(mean) <= tol, (mean, tol)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", [(1, 151936), (8, 151936), (30, 65000), (5, 262144), (12, 40000)])
@pytest.mark.parametrize("n", [1, 20, 64, 100, 128])
def test_top_parts_far_below_each_other(sampler, kind, rows, V, n):
    """Stretches of a row that are forbidden by a large negative number, beside others at -inf and ordinary ones."""
    rng = np.random.default_rng(V + n)
    x = rng.standard_normal((rows, V))
    for r in range(rows):
        for low in rng.permutation([-30.0, -1e4, -1e30, -3.38e38, -np.inf, -np.inf]):
            at, much = rng.integers(0, V), rng.integers(1, V // 3)
            x[r, at:at + much] = low + (rng.standard_normal(len(x[r, at:at + much])) if low == -1e4 else 0)
        x[r, V // 40 * (r % 40):V // 40 * (r % 40) + 200] = rng.standard_normal(200)
    x = _round(x, kind)
    T = rng.choice([0.02, 0.9, 1.0, 1.5], rows).astype(np.float32)
    T[0] = 1.0
    got = _run_top(sampler, x, kind, n, T=T, entropy=False)
    in_range = T >= 1
    _check_top({k: v[in_range] for k, v in got.items()}, x[in_range], n, T=T[in_range])
    assert not np.isnan(got["logprobs"]).any() and not np.isnan(got["rest"]).any()
    assert (got["logprobs"][:, 0] > -20).all()


@pytest.mark.parametrize("n", [1, 20, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_top_lists_at_low_temperatures(sampler, kind, n):
    """Keys that came in before a cut ended, thousands of powers of two below the new reference."""
    rng = np.random.default_rng(n)
    chunk = 8192 if kind == "bf16" else 4096
    rows, V, kinds = 640, 9 * chunk, 24
    x = np.concatenate([_lists_under_way(rng, kinds // 2, V, chunk, first, kind) for first in (5, 6)])
    x[::2, 7 * chunk:] = _round(0.01 * rng.standard_normal(x[::2, 7 * chunk:].shape), kind)  # the cut's list is the last
    x = x[np.arange(rows) * 7 % kinds]
    T = np.float32([0.003, 0.01])[np.arange(rows) // kinds % 2]
    got = _run_top(sampler, x, kind, n, T=T, entropy=False)
    few = {k: v[:2 * kinds] for k, v in got.items()}
    _check_top(few, x[:2 * kinds], n, T=T[:2 * kinds])
    assert not any(np.isnan(v).any() for v in got.values())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", [(1, 151936), (8, 151936), (40, 65000), (20, 262144), (30, 40000)])
@pytest.mark.parametrize("n", [1, 20, 64, 100, 128])
def test_top_most_parts_far_below(sampler, kind, rows, V, n):
    """All that is not forbidden is in one stretch of the row; other parts leave full lists of large negative numbers."""
    rng = np.random.default_rng(V + n)
    x = np.full((rows, V), -np.inf)
    for r in range(rows):
        ends = np.sort(rng.integers(0, V, 5))
        for low, a, b in zip(rng.permutation([-1e4, -1e4, -1e3, -1e30, -np.inf, -3.38e38]), np.append(0, ends), np.append(ends, V)):
            x[r, a:b] = low + (rng.standard_normal(b - a) if low == -1e4 else 0)
        much, at = rng.integers(n, V // 20), rng.integers(0, V)
        x[r, at:at + much] = rng.standard_normal(len(x[r, at:at + much]))
        x[r, rng.integers(0, V)] = 1.0
    x = _round(x, kind)
    got = _run_top(sampler, x, kind, n)
    _check_top(got, x, n)
    _check_rest(got, x, n)


@pytest.mark.parametrize("n", [20, 64, 100])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_top_keys_below_the_reference(sampler, kind, n):
    """While a list is cut more keys come than are cut at once, above the old bar and below what the cut leaves, at temperatures
    by which they are thousands of powers of two below that."""
    rng = np.random.default_rng(n)
    chunk = 8192 if kind == "bf16" else 4096
    rows, V, kinds = 320, 9 * chunk, 32
    x = 0.01 * rng.standard_normal((kinds, V))
    for r in range(kinds):
        first = 5 + r % 2
        lanes, second, third = rng.integers(n // 2, n), rng.integers(n + 60, n + 140), rng.integers(150, 250)
        x[r, rng.permutation(chunk)[:3 * lanes]] = 2 + 0.1 * rng.random(3 * lanes)
        x[r, first * chunk + rng.permutation(chunk)[:second]] = 6 + 3 * rng.random(second)
        x[r, (first + 1) * chunk + rng.permutation(chunk)[:third]] = 2.5 + 3 * rng.random(third)
    x = _round(x, kind)[np.arange(rows) % kinds]
    T = np.float32([0.002, 0.01])[np.arange(rows) // kinds % 2]
    got = _run_top(sampler, x, kind, n, T=T, entropy=False)
    assert not any(np.isnan(v).any() for v in got.values())
    few = {k: v[:2 * kinds] for k, v in got.items()}
    _check_top(few, x[:2 * kinds], n, T=T[:2 * kinds])
    _check_rest(few, x[:2 * kinds], n, T[:2 * kinds])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", [(20, 300), (20, 9000), (8, 151936), (400, 6000)])
def test_top_rest_below_the_range(sampler, kind, rows, V):
    """Tokens forbidden by the type's lowest value, at temperatures by which their logprobs are below fp32's range or not."""
    rng = np.random.default_rng(V)
    x = rng.standard_normal((rows, V))
    x[:, 3 * V // 4:] = -3.3895314e38 if kind == "bf16" else -3.4028235e38
    x[::2, V // 40:3 * V // 4] = -np.inf
    x[::4, :V // 40] = x[0, -1]
    x[::4, 1] = 2.0
    x = _round(x, kind)
    T = rng.choice([0.3, 0.99, 1.0, 1.1, 3.0], rows).astype(np.float32)
    for n in (1, V // 40, 128):
        if n <= 128:
            got = _run_top(sampler, x, kind, n, V % 3, V % 5, T=T, entropy=False)
            _check_rest(got, x, n, T)
            assert not np.isnan(got["logprobs"]).any()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", [(320, 14000), (40, 3000), (320, 60000), (3, 262144)])
@pytest.mark.parametrize("entropy", [True, False])
def test_top_sums_of_few_different_values(sampler, kind, rows, V, entropy):
    """Sums whose terms are alike, so that their roundings are."""
    rng = np.random.default_rng(V)
    V = V if kind == "bf16" else V // 2
    kinds = 24
    x = rng.integers(0, rng.integers(2, 8, (kinds, 1)), (kinds, V)) * rng.choice([0.3, 0.5, 0.7], (kinds, 1))
    x[:, V // 3] = rng.uniform(4, 9, kinds)
    for r in range(0, kinds, 2):  # two values, of which more have the larger one than a list holds
        x[r] = 0
        x[r, rng.permutation(V)[:rng.integers(300, 1200)]] = rng.choice([2.0, 4.0, 6.0, 7.0])
    x[::4], x[::4, :1024] = 0, 6.0
    x = _round(x, kind)[np.arange(rows) % kinds]
    T = rng.choice([0.7, 0.9, 1.3], rows).astype(np.float32)
    T[::4] = 1.0
    for n in (1, 20):
        got = _run_top(sampler, x, kind, n, T=T, entropy=entropy)
        some = np.arange(min(rows, 48))
        _check_top({k: v[some] for k, v in got.items()}, x[some], n, T=T[some])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [2, 400, 9000, 60000, 200000])
def test_distill_infinite_divergences(sampler, kind, V):
    """Lists of which the student forbids all tokens of a part of the row, or all, at temperatures below 1 and above."""
    k = min(10, V)
    for coef in (0.0, 0.3):
        b = Batch(V, 12, V, k, kind, coef=coef)
        b.T = np.float32([0.7, 0.9, 0.99, 1.0, 1.5, 30.0] * 2)
        b.tokens[:] = b.ids[:, 0] if V > 2 else V - 1
        if V > 2:
            b.tokens[:] = np.array([np.setdiff1d(np.arange(40), b.ids[r])[0] for r in range(12)])
        for r in range(12):
            some = b.ids[r] if r < 6 and V > 2 else b.ids[r, -1:]
            some = some[some != b.tokens[r]]
            b.x[r, some] = -np.inf
            b.x[r, b.tokens[r]] = 1.0
        b.run(sampler, scale=0.7).check()
        want = O.distill(b.x, b.ids, b.l, b.rest, b.tokens, coef, b.T, b.weight)
        if V > 2:
            assert np.isinf(want["kl"]).all() and np.isinf(want["loss"])


@pytest.mark.parametrize("rows,V,kind", [(170, 40000, "bf16"), (60, 100001, "f32"), (40, 200000, "f32"), (90, 151937, "bf16"),
                                         (60, 128000, "f32"), (400, 20011, "f32"), (30, 262144, "bf16")])
def test_distill_without_gradient_on_clusters_of_all_sizes(sampler, rows, V, kind):
    """Parts of up to three steps in two buffers, several rows for each cluster."""
    b = Batch(V, rows, V, 30, kind, pad=V % 3, shift=V % 5, heat=True, kept=0.9, coef=0.1, short=0.3)
    b.run(sampler, grad=False).check()
