"""Scoring and the losses on the GPU against their definitions in double
precision (oracle/losses.py). Needs a GB300.

Tolerances, from the kernels' fp32 arithmetic (eps = 2^-24, one rounding). With
y = x / T in nats and m the row's largest y:
 - an exponential's argument carries the rounding of log2(e) / T (the constant
   and the division), of the difference and of the product times |y - m|: three
   roundings of a full half step between them, and 2^-22 of the exponential
   itself;
 - a sum of A terms one after another, rounded at random, is within 4 sqrt(A)
   eps of itself (the probabilistic bound of Higham and Mary with lambda = 4);
   A is at most V / 256 + 64 in a thread and the joins after it;
 - references inside a row may differ by 6 nats;
 - every output has its own rounding, half a step of its type.
"""
import numpy as np
import pytest

import oracle.losses as L
import workloads

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def sampler():
    from decode_step_token_gb300 import build
    build.build_library()
    import decode_step_token_gb300 as d
    s = d.Sampler(max_rows=2048, max_vocab=262144)
    yield s
    s.close()


class Rows:
    """Inputs of n rows on both sides, and the outputs' buffers."""

    def __init__(self, seed, n, V, kind="f32", pad=0, shift=0, heat=False, kept=1.0, banned=0.0, grad=True,
                 grad_pad=None, grad_shift=0, scale=2.0):
        import torch

        rng = np.random.default_rng(seed)
        self.n, self.V, self.kind, self.rng = n, V, kind, rng
        x = (scale * rng.standard_normal((n, V))).astype(np.float32)
        self.tokens = rng.integers(0, V, n).astype(np.int32)
        rows = np.arange(n)
        if banned:
            x[rng.random((n, V)) < banned] = -np.inf
        x[rows, self.tokens] = rng.uniform(0, 9, n)
        self.weight = None
        if kept < 1.0:
            self.weight = rng.uniform(0.25, 1.0, n).astype(np.float32)
            self.weight[rng.permutation(n)[:int(round((1 - kept) * n))]] = 0
            x[self.weight == 0] = np.nan  # what a left-out row holds is not read
        self.T = rng.uniform(0.5, 1.6, n).astype(np.float32) if heat else None
        if kind == "bf16":
            x = workloads.bf16_bits_to_f32(workloads.to_bf16_bits(x)).reshape(n, V)
        self.x = x
        self.torch_type = torch.bfloat16 if kind == "bf16" else torch.float32
        self.pad, self.shift = pad, shift
        self.grad_pad = pad if grad_pad is None else grad_pad
        self.grad_shift = grad_shift
        self.want_grad = grad
        self.upload()

    def _buffer(self, pad, shift, fill):
        import torch

        flat = torch.full((self.n * (self.V + pad) + shift + 64,), fill, dtype=self.torch_type, device="cuda:0")
        return flat, flat[shift:shift + self.n * (self.V + pad)].view(self.n, self.V + pad)[:, :self.V]

    def upload(self):
        import torch

        def dev(a):
            return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")

        # the values between the rows and beside them must not matter
        self.flat, self.logits = self._buffer(self.pad, self.shift, float("nan"))
        self.logits.copy_(torch.from_numpy(self.x))
        self.d_tokens, self.d_T, self.d_w = dev(self.tokens), dev(self.T), dev(self.weight)
        self.gflat, self.grad = self._buffer(self.grad_pad, self.grad_shift, -7.0) if self.want_grad else (None, None)
        self.out = {k: torch.full((self.n,), -7.0, device="cuda:0") for k in ("logprob", "entropy", "ratio", "kl")}
        self.status = torch.full((self.n,), -7, dtype=torch.int32, device="cuda:0")
        self.loss = torch.full((1,), -7.0, device="cuda:0")

    def kw(self):
        return dict(logits=self.logits, tokens=self.d_tokens, temperature=self.d_T, weight=self.d_w,
                    out_logprob=self.out["logprob"], out_status=self.status)

    def host(self, name):
        return self.out[name].double().cpu().numpy()

    # ------------------------------------------------------------------ tolerances
    def tolerances(self, got):
        t = {k: np.zeros(self.n) for k in ("s", "logprob", "entropy")}
        adds = 4.0 * np.sqrt(self.V / 256 + 64) * EPS
        for r in np.nonzero((got["status"] == 0) & (self.live()))[0]:
            logp = got["logp"][r]
            p, depth = np.exp(logp), np.where(np.isfinite(logp), logp.max() - logp, 0.0)
            near = (p * depth).sum()
            t["s"][r] = 2.0 ** -22 + 3 * EPS * near + adds
            t["logprob"][r] = (t["s"][r] + 3 * EPS * min(depth[self.tokens[r]], 1e4) + EPS * abs(got["logprob"][r])
                               + 2 * EPS)
            far = near + 6.0
            t["entropy"][r] = (t["s"][r] * (1 + far) + far * (2.0 ** -22 + adds + 4 * EPS)
                               + 3 * EPS * 2 * ((p * depth ** 2).sum() + 36) + EPS * abs(got["entropy"][r]))
        return t

    def live(self):
        return np.ones(self.n, bool) if self.weight is None else self.weight != 0

    def check_rows(self, got, entropy=True):
        tol = self.tolerances(got)
        np.testing.assert_array_equal(self.status.cpu().numpy(), got["status"])
        for name in ("logprob", "entropy")[:2 if entropy else 1]:
            a, b = self.host(name), got[name]
            b = np.where(np.abs(b) > np.finfo(np.float32).max, np.copysign(np.inf, b), b)  # as fp32 holds it
            assert np.array_equal(np.isnan(a), np.isnan(b)), name
            fine = np.isfinite(b)
            assert np.array_equal(a[~fine & ~np.isnan(b)], b[~fine & ~np.isnan(b)]), name
            bad = np.abs(a[fine] - b[fine]) > tol[name][fine]
            assert not bad.any(), (name, np.nonzero(bad)[0][:5], a[fine][bad][:5], b[fine][bad][:5])
        return tol

    def check_grad(self, got, tol, by_lp, tol_lp, by_h=None, tol_h=None):
        """by_lp, by_h: the exact gradients by the logprob and the entropy, with their errors."""
        import torch

        g = self.grad.double().cpu().numpy()
        beside = torch.ones_like(self.gflat, dtype=torch.bool)
        beside[self.grad_shift:self.grad_shift + self.n * (self.V + self.grad_pad)].view(
            self.n, -1)[:, :self.V] = False
        assert bool((self.gflat[beside] == -7.0).all()), "written beside the gradient"
        want = got["grad"]
        for r in range(self.n):
            nan = np.isnan(want[r])
            assert np.array_equal(np.isnan(g[r]), nan), r
            if nan.all() or not self.live()[r] or got["status"][r] != 0:
                assert nan.all() or (g[r] == 0).all(), r
                continue
            T = 1.0 if self.T is None or self.T[r] < 1e-5 else float(self.T[r])
            logp = got["logp"][r]
            p = np.exp(logp)
            depth = np.where(p > 0, logp.max() - logp, 0.0)
            lnp = np.where(p > 0, logp, 0.0)
            a, da = abs(by_lp[r]), tol_lp[r]
            b, db = (abs(by_h[r]), 0.0 if tol_h is None else tol_h[r]) if by_h is not None else (0.0, 0.0)
            rel = 2.0 ** -22 + 3 * EPS * depth + tol["s"][r] + 6 * EPS
            size = a + b * np.abs(lnp + got["entropy"][r])
            # k0 + k1 u joins terms of the size of b (|ln p| + entropy + ln s)
            parts = a + b * (np.abs(lnp) + abs(got["entropy"][r]) + 2 * np.log(self.V + 1) + 8)
            err = p / T * (rel * size + 8 * EPS * parts + da + db * np.abs(lnp + got["entropy"][r])
                           + b * (tol["entropy"][r] + tol["s"][r] + 3 * EPS * depth))
            err[self.tokens[r]] += (da + 4 * EPS * a) / T
            lim = HALF[self.kind] * np.abs(want[r]) + err * (1 + HALF[self.kind]) + 1e-37
            bad = np.abs(g[r] - want[r]) > lim
            assert not bad.any(), (r, np.nonzero(bad)[0][:5], g[r][bad][:5], want[r][bad][:5], lim[bad][:5])


# one token, one element, widths around the vector's 8 and 4, around a warp's and a block's share, odd
# widths, the vocabularies of the framework's workloads; rows and gradients that start off a 16-byte boundary
SHAPES = [
    dict(n=1, V=1), dict(n=3, V=2, kind="bf16"), dict(n=5, V=7, kind="bf16", pad=1),
    dict(n=4, V=8, kind="bf16"), dict(n=4, V=9, pad=3, shift=1), dict(n=9, V=255, kind="bf16", shift=3),
    dict(n=33, V=1000, heat=True, kept=0.7), dict(n=160, V=1024, kind="bf16", heat=True, banned=0.3),
    dict(n=17, V=4097, kind="bf16", pad=2, shift=5, grad_pad=4, grad_shift=1, kept=0.5),
    dict(n=6, V=4096, kind="bf16", grad_shift=8), dict(n=6, V=4096, grad_shift=2),
    dict(n=40, V=17001, heat=True, banned=0.5), dict(n=3, V=40961, kind="bf16", pad=7, heat=True),
    dict(n=1, V=128000, kind="bf16"), dict(n=9, V=128000, heat=True, kept=0.8, shift=2),
    dict(n=20, V=151936, kind="bf16", heat=True), dict(n=2, V=262144, heat=True), dict(n=2, V=262144, kind="bf16"),
    dict(n=700, V=3000, kind="bf16", kept=0.9), dict(n=320, V=20011, kind="bf16", heat=True, kept=0.9, pad=5),    # few rows in the registers of a block of 8 and 16 warps, and few longer ones
    dict(n=5, V=9001, kind="bf16", pad=3, shift=1), dict(n=150, V=32000, kind="bf16", kept=0.8, heat=True),
    dict(n=60, V=16001, kept=0.5, banned=0.3), dict(n=13, V=151936, kind="bf16", pad=3, shift=1, kept=0.7, heat=True),
    dict(n=7, V=100003, banned=0.5, pad=1, grad_pad=2), dict(n=50, V=40961, kind="bf16", heat=True),
    dict(n=14, V=65537, kind="bf16", grad_shift=3, kept=0.6),
]
# several rows for each cluster, at every way of cutting a row: one CTA a row and more, parts of which two fit in
# the ring and parts of which one does, rows in registers
MANY = [
    dict(n=650, V=9001, kind="bf16", kept=0.6), dict(n=330, V=32000, kind="bf16"),
    dict(n=170, V=64000, kind="bf16", kept=0.5, heat=True), dict(n=100, V=128000, kind="bf16", kept=0.8),
    dict(n=90, V=151936, kind="bf16", pad=3, shift=1), dict(n=50, V=128000, kept=0.9), dict(n=40, V=200003, pad=1),
    dict(n=900, V=1500, kept=0.5), dict(n=300, V=5000, kind="bf16", banned=0.3), dict(n=300, V=4001, shift=3),
]


def _id(s):
    return "-".join(f"{k}{v}" for k, v in s.items())


@pytest.mark.parametrize("shape", SHAPES, ids=_id)
def test_score(sampler, shape):
    c = Rows(1, grad=False, **shape)
    sampler.score(out_entropy=c.out["entropy"], **c.kw())
    c.check_rows(L.score(c.x, c.tokens, c.T, c.weight))


@pytest.mark.parametrize("shape", SHAPES, ids=_id)
@pytest.mark.parametrize("entropy", [False, True])
def test_score_grad(sampler, shape, entropy):
    import torch

    c = Rows(2, **shape)
    a = c.rng.standard_normal(c.n).astype(np.float32)
    b = c.rng.standard_normal(c.n).astype(np.float32) if entropy else None
    sampler.score_grad(grad_logprob=torch.from_numpy(a).cuda(), out_grad=c.grad, out_entropy=c.out["entropy"],
                       grad_entropy=torch.from_numpy(b).cuda() if entropy else None, **c.kw())
    got = L.score(c.x, c.tokens, c.T, c.weight)
    tol = c.check_rows(got)
    got["grad"] = L.logits_grad(got, c.tokens, a.astype(np.float64), b, c.T, c.weight)
    c.check_grad(got, tol, a, np.zeros(c.n), b)


@pytest.mark.parametrize("shape", MANY, ids=_id)
@pytest.mark.parametrize("mode", ["score", "clip", "entropy"])
def test_many_rows(sampler, shape, mode):
    import torch

    c = Rows(12, grad=mode != "score", **shape)
    if mode == "score":
        sampler.score(**c.kw())
        c.check_rows(L.score(c.x, c.tokens, c.T, c.weight), entropy=False)
        return
    a = c.rng.standard_normal(c.n).astype(np.float32)
    b = c.rng.standard_normal(c.n).astype(np.float32) if mode == "entropy" else None
    sampler.score_grad(grad_logprob=torch.from_numpy(a).cuda(), out_grad=c.grad,
                       out_entropy=c.out["entropy"] if b is not None else None,
                       grad_entropy=torch.from_numpy(b).cuda() if b is not None else None, **c.kw())
    got = L.score(c.x, c.tokens, c.T, c.weight)
    tol = c.check_rows(got, entropy=b is not None)
    got["grad"] = L.logits_grad(got, c.tokens, a.astype(np.float64), b, c.T, c.weight)
    c.check_grad(got, tol, a, np.zeros(c.n), b)


def policy_inputs(c, got):
    """Old logprobs whose ratios lie on both sides of the clips, at least 1 % away from them."""
    choices = np.log(np.array([0.3, 0.7, 0.85, 1.0, 1.1, 1.24, 1.4, 3.0]))
    lp = np.where(np.isfinite(got["logprob"]), got["logprob"], 0.0)
    old = (lp - c.rng.choice(choices, c.n)).astype(np.float32)
    adv = np.where(c.rng.random(c.n) < 0.1, 0.0, c.rng.standard_normal(c.n)).astype(np.float32)
    ref = (lp + c.rng.choice([1e-4, 0.1, 0.49, 0.51, 2.0], c.n) * c.rng.choice([-1, 1], c.n)).astype(np.float32)
    return old, adv, ref


@pytest.mark.parametrize("shape", SHAPES, ids=_id)
@pytest.mark.parametrize("terms", ["clip", "kl", "entropy"])
def test_policy_loss(sampler, shape, terms):
    import torch

    c = Rows(3, **shape)
    old, adv, ref = policy_inputs(c, L.score(c.x, c.tokens, c.T, c.weight))
    kl, ent = (0.07 if terms != "clip" else 0.0), (0.03 if terms == "entropy" else 0.0)
    kw = dict(clip_low=0.25, clip_high=0.3, kl_coef=kl, entropy_coef=ent)
    cu = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    ins = dict(old_logprob=cu(old), advantage=cu(adv), ref_logprob=cu(ref) if kl else None, out_loss=c.loss,
               out_ratio=c.out["ratio"], out_kl=c.out["kl"] if kl else None, out_entropy=c.out["entropy"])
    sampler.policy_loss(grad_scale=0.5, grad_scale_dev=torch.tensor([3.0], device="cuda:0"), out_grad=c.grad, **ins,
                        **kw, **c.kw())
    got = L.policy(c.x, c.tokens, old.astype(np.float64), adv.astype(np.float64),
                   ref.astype(np.float64) if kl else None, c.T, c.weight, grad_scale=1.5, **kw)
    tol = c.check_rows(got)
    w = np.ones(c.n) if c.weight is None else c.weight.astype(np.float64)
    live = c.live()
    # the clips' bounds and every product are rounded once; exp has 2 eps of its own
    t_ratio = got["ratio"] * (tol["logprob"] + EPS * np.abs(got["logprob"] - old) + 6 * EPS)
    t_term = t_ratio * np.abs(adv) + 8 * EPS * np.abs(got["ratio"] * adv)
    t_by = t_term.copy()
    t_kl = np.zeros(c.n)
    if kl:
        d = ref - got["logprob"]
        t_d = tol["logprob"] + EPS * np.abs(d)
        # from 1/2 on the KL is a difference of two rounded values
        t_kl = (np.abs(np.expm1(d)) * t_d + 0.5 * np.exp(np.abs(d)) * t_d ** 2
                + 8 * EPS * (got["kl"] + (np.abs(d) >= 0.49) * (np.abs(np.expm1(d)) + np.abs(d))))
        t_term += kl * t_kl
        t_by += kl * (np.exp(d) * t_d + 8 * EPS * np.abs(np.expm1(d)))
    if ent:
        t_term += ent * (tol["entropy"] + 4 * EPS * got["entropy"])

    def check_outputs():
        assert (np.abs(c.host("ratio") - got["ratio"]) <= t_ratio).all()
        if kl:
            assert (np.abs(c.host("kl") - got["kl"])[live] <= t_kl[live]).all()
            assert (c.host("kl")[~live] == 0).all()
        assert abs(c.loss.item() - got["loss"]) <= (w * t_term)[live].sum() + 2 * EPS * abs(got["loss"])

    check_outputs()
    c.check_grad(got, tol, got["by_logprob"], 1.5 * w * (t_by + 4 * EPS * np.abs(got["by_logprob"])),
                 got["by_entropy"])
    # without the gradient: the same outputs
    for v in (c.loss, *c.out.values()):
        v.fill_(-7.0)
    sampler.policy_loss(**ins, **kw, **c.kw())
    c.check_rows(got)
    check_outputs()


@pytest.mark.parametrize("shape", [dict(n=9, V=7, kind="bf16", pad=1), dict(n=40, V=1000, kept=0.6, heat=True),
                                   dict(n=300, V=3001, kind="bf16", kept=0.7, shift=3),
                                   dict(n=24, V=128000, kind="bf16", kept=0.8), dict(n=11, V=40961, banned=0.3)],
                         ids=_id)
@pytest.mark.parametrize("mean,smooth,margin,with_ref", [(False, 0.0, 0.0, True), (True, 0.1, 0.5, False),
                                                         (False, 1.0, 0.2, True)])
def test_preference_loss(sampler, shape, mean, smooth, margin, with_ref):
    import torch

    c = Rows(4, **shape)
    lp = L.score(c.x, c.tokens, c.T, c.weight)["logprob"]
    ref = (lp + 0.3 * c.rng.standard_normal(c.n)).astype(np.float32) if with_ref else None
    pairs = 3
    inner = np.sort(c.rng.integers(1, c.n, 2 * pairs - 1))
    offsets = np.concatenate([[1], inner, [c.n - 1]]).astype(np.int32)  # rows 0 and n-1 are in none
    offsets[3] = offsets[2]  # an empty answer
    beta = 0.4
    reward = torch.full((2 * pairs,), -7.0, device="cuda:0")
    kw = dict(beta=beta, margin=margin, label_smoothing=smooth, mean_over_tokens=mean)
    sampler.preference_loss(seq_offsets=torch.from_numpy(offsets).cuda(), out_loss=c.loss, out_reward=reward,
                            ref_logprob=None if ref is None else torch.from_numpy(ref).cuda(), out_grad=c.grad,
                            grad_scale=2.0, grad_scale_dev=torch.tensor([0.25], device="cuda:0"), **kw, **c.kw())
    got = L.preference(c.x, c.tokens, offsets, None if ref is None else ref.astype(np.float64), c.T, c.weight,
                       grad_scale=0.5, **kw)
    tol = c.check_rows(got, entropy=False)
    w = np.ones(c.n) if c.weight is None else c.weight.astype(np.float64)
    t_reward = np.zeros(2 * pairs)
    share = np.ones(2 * pairs)
    for s in range(2 * pairs):
        at = slice(offsets[s], offsets[s + 1])
        share[s] = 1.0 / w[at].sum() if mean and w[at].sum() else 1.0
        t_reward[s] = beta * share[s] * ((w * tol["logprob"])[at]).sum() + 2 * EPS * abs(got["reward"][s])
    assert (np.abs(reward.double().cpu().numpy() - got["reward"]) <= t_reward).all()
    # beta, the margin and the smoothing are floats
    t_z = t_reward[0::2] + t_reward[1::2] + EPS * (np.abs(got["reward"]).max() + margin + 1)
    assert abs(c.loss.item() - got["loss"]) <= t_z.sum() / pairs + 4 * EPS * (1 + abs(got["loss"]))
    t_by = np.zeros(c.n)
    for s in range(2 * pairs):  # sigmoid has a slope of at most 1/4
        at = slice(offsets[s], offsets[s + 1])
        t_by[at] = 0.5 * w[at] * beta * share[s] / pairs * (t_z[s // 2] / 4 + EPS)
    c.check_grad(got, tol, got["by_logprob"], t_by + 8 * EPS * np.abs(got["by_logprob"]))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_status_rows(sampler, kind):
    """Rows with an error report it and take NaN; the others keep their values."""
    import torch

    c = Rows(5, 12, 3001, kind, heat=True)
    c.x[1, 5], c.x[2, 3000], c.x[3], c.x[4, 7] = np.nan, np.inf, -np.inf, -np.inf
    c.tokens[5], c.tokens[6] = 3001, -1
    c.T[7], c.T[8], c.T[9], c.T[10] = np.nan, -1.0, np.inf, 5e-6
    c.x[11, :] = -np.inf
    c.x[11, c.tokens[11]] = -1e30  # the only token there is
    if kind == "bf16":
        c.x = workloads.bf16_bits_to_f32(workloads.to_bf16_bits(c.x)).reshape(c.n, c.V)
    c.upload()
    got = L.score(c.x, c.tokens, c.T, None)
    assert got["status"].tolist() == [0, 1, 1, 2, 0, 3, 3, 3, 3, 3, 0, 0]
    a = np.ones(c.n, np.float32)
    sampler.score_grad(grad_logprob=torch.from_numpy(a).cuda(), out_grad=c.grad, out_entropy=c.out["entropy"],
                       **c.kw())
    tol = c.check_rows(got)
    got["grad"] = L.logits_grad(got, c.tokens, a, None, c.T)
    c.check_grad(got, tol, a, np.zeros(c.n))
    # a loss with such a row is NaN, and not because of a row that is left out
    zeros = torch.zeros(c.n, device="cuda:0")
    sampler.policy_loss(old_logprob=zeros, advantage=zeros, out_loss=c.loss, **c.kw())
    assert torch.isnan(c.loss).item()
    c.weight = (got["status"] == 0).astype(np.float32)
    c.upload()
    sampler.policy_loss(old_logprob=zeros, advantage=zeros, out_loss=c.loss, **c.kw())
    assert c.loss.item() == 0.0
    assert (c.status.cpu().numpy() == 0).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_extreme_values(sampler, kind):
    """Masks of the type's lowest value, one token with all the mass, flat rows, a
    token without mass, and temperatures near the greedy threshold."""
    import torch

    c = Rows(6, 8, 5003, kind, heat=True)
    low = float(torch.finfo(c.torch_type).min)
    c.x[0, :] = low
    c.x[0, c.tokens[0]] = 3.0
    c.x[1, :] = low          # nothing but the lowest value: a flat row
    c.x[2, :] = 1e30
    c.x[3, :] = 0.0
    c.x[3, 17] = 200.0
    c.T[4] = 2e-5
    c.T[5] = 1e4
    c.x[6, c.tokens[6]] = -np.inf
    c.x[7, 1::2] = low
    if kind == "bf16":
        c.x = workloads.bf16_bits_to_f32(workloads.to_bf16_bits(c.x)).reshape(c.n, c.V)
    c.upload()
    got = L.score(c.x, c.tokens, c.T, None)
    assert got["logprob"][6] == -np.inf and (got["status"] == 0).all()
    a, b = np.ones(c.n, np.float32), np.full(c.n, 0.5, np.float32)
    sampler.score_grad(grad_logprob=torch.from_numpy(a).cuda(), grad_entropy=torch.from_numpy(b).cuda(),
                       out_grad=c.grad, out_entropy=c.out["entropy"], **c.kw())
    tol = c.check_rows(got)
    got["grad"] = L.logits_grad(got, c.tokens, a, b, c.T)
    c.check_grad(got, tol, a, np.zeros(c.n), b)


@pytest.mark.parametrize("kind,n,V", [("f32", 5, 1003), ("bf16", 400, 20011), ("bf16", 3, 128000)])
def test_gradient_in_place(sampler, kind, n, V):
    import torch

    c = Rows(7, n, V, kind, kept=0.7)
    a = torch.from_numpy(c.rng.standard_normal(n).astype(np.float32)).cuda()
    sampler.score_grad(grad_logprob=a, out_grad=c.grad, **c.kw())
    apart = c.grad.clone()
    sampler.score_grad(grad_logprob=a, out_grad=c.logits, **c.kw())
    assert torch.equal(c.logits, apart)
    c.upload()
    ends = torch.tensor([0, n // 2, n], dtype=torch.int32, device="cuda:0")
    sampler.preference_loss(seq_offsets=ends, out_loss=c.loss, out_grad=c.grad, **c.kw())
    apart = c.grad.clone()
    sampler.preference_loss(seq_offsets=ends, out_loss=c.loss, out_grad=c.logits, **c.kw())
    assert torch.equal(c.logits, apart)


@pytest.mark.parametrize("V,kind", [(33, "bf16"), (70, "f32"), (20011, "bf16")])
def test_forbidden_tokens_at_many_temperatures(sampler, V, kind):
    """-inf logits (and the elements of a row's neighbours that its first and last vectors hold) stay without
    mass at every temperature: the factor log2(e) / T is a pair, whose parts have to have the same sign."""
    import torch

    n = 2048
    gen = torch.Generator(device="cuda:0").manual_seed(2)
    x = torch.randn((n, V), generator=gen, device="cuda:0").to(torch.bfloat16 if kind == "bf16" else torch.float32)
    x[:, 1::3] = -torch.inf
    T = 10.0 ** (6.0 * torch.rand(n, generator=gen, device="cuda:0") - 2.0)
    tok = torch.zeros(n, dtype=torch.int32, device="cuda:0")
    lp, ent = torch.empty(n, device="cuda:0"), torch.empty(n, device="cuda:0")
    sampler.score(logits=x, tokens=tok, temperature=T, out_logprob=lp, out_entropy=ent)
    want = torch.log_softmax(x.double() / T.double()[:, None], 1)[:, 0]
    # see the tolerances above: the depth of a token at T = 0.01 is up to 800 nats
    tol = 2.0 ** -22 + 3 * EPS * want.abs() * 2 + 4 * (V / 256 + 64) ** 0.5 * EPS + EPS * want.abs() + 2 * EPS
    assert torch.isfinite(lp).all() and torch.isfinite(ent).all()
    assert ((lp.double() - want).abs() <= tol).all()


def test_same_bits_each_time_and_in_a_graph(sampler):
    import torch

    c = Rows(8, 500, 9001, "bf16", kept=0.8, heat=True)
    old = torch.from_numpy(c.rng.normal(-3, 1, c.n).astype(np.float32)).cuda()
    adv = torch.from_numpy(c.rng.standard_normal(c.n).astype(np.float32)).cuda()
    ends = torch.tensor([0, 120, 250, 260, 499], dtype=torch.int32, device="cuda:0")
    grad2, loss2 = torch.empty_like(c.grad), torch.empty_like(c.loss)

    def both(stream):
        sampler.policy_loss(old_logprob=old, advantage=adv, ref_logprob=old, kl_coef=0.1, out_loss=c.loss,
                            out_grad=c.grad, stream=stream, **c.kw())
        sampler.preference_loss(seq_offsets=ends, ref_logprob=old, out_loss=loss2, out_grad=grad2, stream=stream,
                                **c.kw())

    def seen():
        torch.cuda.synchronize()
        return [t.clone() for t in (c.loss, c.grad, c.out["logprob"], loss2, grad2)]

    both(None)
    first = seen()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        both(side.cuda_stream)
    for a, b in zip(first, seen()):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both(torch.cuda.current_stream().cuda_stream)
    for t in (c.loss, c.grad, loss2, grad2):
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(2):
        graph.replay()
    for a, b in zip(first, seen()):
        assert torch.equal(a, b)


def test_nothing_to_do(sampler):
    import torch

    x = torch.empty((0, 100), device="cuda:0")
    tok = torch.empty(0, dtype=torch.int32, device="cuda:0")
    none = torch.empty(0, device="cuda:0")
    loss = torch.full((1,), -7.0, device="cuda:0")
    sampler.score(logits=x, tokens=tok)
    sampler.policy_loss(logits=x, tokens=tok, old_logprob=none, advantage=none, out_loss=loss)
    assert loss.item() == 0.0
    reward = torch.full((2,), -7.0, device="cuda:0")
    ends = torch.zeros(3, dtype=torch.int32, device="cuda:0")
    sampler.preference_loss(logits=x, tokens=tok, seq_offsets=ends, out_loss=loss, out_reward=reward)
    assert abs(loss.item() - np.log(2)) < 1e-7 and (reward == 0).all()
    c = Rows(9, 4, 50)
    sampler.preference_loss(seq_offsets=ends[:1], out_loss=c.loss, out_grad=c.grad, **c.kw())
    assert c.loss.item() == 0.0 and (c.grad == 0).all()


@pytest.mark.parametrize("bad", [[0, 3, 9, 5, 10], [-1, 3, 5, 8, 10], [0, 3, 5, 8, 2 ** 30]])
def test_bad_offsets(sampler, bad):
    """Answers that do not lie within the rows: NaN, and nothing read or written out of bounds."""
    import torch

    c = Rows(10, 10, 301)
    reward = torch.full((4,), -7.0, device="cuda:0")
    sampler.preference_loss(seq_offsets=torch.tensor(bad, dtype=torch.int32, device="cuda:0"), out_loss=c.loss,
                            out_reward=reward, out_grad=c.grad, **c.kw())
    ok = [0 <= bad[s] <= bad[s + 1] <= 10 for s in range(4)]
    assert torch.isnan(c.loss).item() and torch.isnan(reward).tolist() == [not v for v in ok]


def test_refusals(sampler):
    import torch
    import decode_step_token_gb300 as d

    c = Rows(11, 4, 64)
    v = torch.zeros(4, device="cuda:0")

    def code(f, **kw):
        with pytest.raises(d.SamplerError) as e:
            f(**{**c.kw(), **kw})
        return e.value.code

    pol = dict(old_logprob=v, advantage=v, out_loss=c.loss)
    for name, val in (("clip_low", -0.1), ("clip_low", 1.1), ("clip_high", -1.0), ("clip_high", float("nan")),
                      ("kl_coef", float("inf")), ("grad_scale", float("nan"))):
        assert code(sampler.policy_loss, **{**pol, name: val}) == -9, name
    assert code(sampler.policy_loss, kl_coef=0.1, **pol) == -1
    assert code(sampler.policy_loss, out_kl=v, **pol) == -1
    ends = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda:0")
    assert code(sampler.preference_loss, seq_offsets=ends, out_loss=c.loss, label_smoothing=1.5) == -9
    with pytest.raises(ValueError, match="pairs"):
        sampler.preference_loss(seq_offsets=ends[:2], out_loss=c.loss, **c.kw())
    with pytest.raises(ValueError, match="out_grad"):
        sampler.score_grad(grad_logprob=v, out_grad=c.grad[:3], **c.kw())
    with pytest.raises(ValueError, match="grad_logprob"):
        sampler.score_grad(grad_logprob=v[:3], out_grad=c.grad, **c.kw())
    with pytest.raises(TypeError, match="tokens"):
        sampler.score(**{**c.kw(), "tokens": c.d_tokens.long()})
    wide = torch.zeros((1, 262145), device="cuda:0")
    with pytest.raises(d.SamplerError) as e:
        sampler.score(logits=wide, tokens=c.d_tokens[:1])
    assert e.value.code == -3
    many = torch.zeros((2049, 8), device="cuda:0")
    with pytest.raises(d.SamplerError) as e:
        sampler.score(logits=many, tokens=torch.zeros(2049, dtype=torch.int32, device="cuda:0"))
    assert e.value.code == -3


def test_agrees_with_the_sampler(sampler):
    """The logprob of a sampled token is the one that the sampler reported for it."""
    import torch

    n, V = 32, 20011
    x = (2.5 * torch.randn((n, V), device="cuda:0")).to(torch.bfloat16)
    T = torch.linspace(0.0, 1.4, n, device="cuda:0")
    tok = torch.empty(n, dtype=torch.int32, device="cuda:0")
    said, ours = torch.empty(n, device="cuda:0"), torch.empty(n, device="cuda:0")
    args = sampler.make_args(logits=x, temperature=T, out_tokens=tok)
    sampler.sample_ex_args(args, out_token_logprob=said)
    sampler.score(logits=x, tokens=tok, temperature=T, out_logprob=ours)
    # the sampler's logprobs are within 1e-6 + 1e-5 |lp| of the exact ones, ours within about 1e-5
    assert ((said - ours).abs() <= 2e-5 + 1e-5 * ours.abs()).all()


@pytest.mark.parametrize("kind,n,V", [("f32", 300, 40961), ("bf16", 40, 151936)])
def test_waits_that_give_up(sampler, kind, n, V):
    """On a handle whose waits give up at once, every row that counts says so and nothing looks like a result:
    outputs, rewards, losses and gradients are NaN, also where an earlier call has left sums in the workspace."""
    import torch
    import decode_step_token_gb300 as d

    old, ends = torch.zeros(n, device="cuda:0"), torch.tensor([0, n // 3, n - 1], dtype=torch.int32, device="cuda:0")
    reward = torch.full((2,), -7.0, device="cuda:0")
    ones = torch.ones(n, device="cuda:0")

    def calls(s, c):
        yield "score", lambda: s.score(out_entropy=c.out["entropy"], **c.kw())
        yield "grad", lambda: s.score_grad(grad_logprob=ones, grad_entropy=ones, out_grad=c.grad, **c.kw())
        yield "policy", lambda: s.policy_loss(old_logprob=old, advantage=ones, ref_logprob=old, kl_coef=0.1,
                                              out_kl=c.out["kl"], out_ratio=c.out["ratio"], out_loss=c.loss,
                                              out_grad=c.grad, **c.kw())
        yield "forward", lambda: s.policy_loss(old_logprob=old, advantage=ones, out_loss=c.loss, **c.kw())
        yield "pairs", lambda: s.preference_loss(seq_offsets=ends, out_loss=c.loss, out_reward=reward, out_grad=c.grad,
                                                 **c.kw())
        yield "pairs forward", lambda: s.preference_loss(seq_offsets=ends, out_loss=c.loss, out_reward=reward, **c.kw())

    with d.Sampler(max_rows=n, max_vocab=V, short_waits=True) as short:
        # rows that stay in registers have no waits: this call leaves its sums and records behind
        few = Rows(13, n, 900, kind)
        short.preference_loss(seq_offsets=ends, out_loss=few.loss, out_reward=reward, out_grad=few.grad, **few.kw())
        assert torch.isfinite(few.loss).all() and torch.isfinite(few.grad).all() and (few.status == 0).all()
        c = Rows(14, n, V, kind, pad=1, kept=0.8)
        live = torch.from_numpy(c.live()).cuda()
        for name, call in calls(short, c):
            for t in (c.loss, c.gflat, *c.out.values(), reward):
                t.fill_(-7.0)
            c.status.fill_(-7)
            call()
            assert torch.equal(c.status, torch.where(live, 5, 0).int()), name
            for k, t in c.out.items():
                if not bool((t == -7).all()):  # not asked of this call
                    assert torch.isnan(t[live]).all() and (t[~live] == 0).all(), (name, k)
            assert torch.isnan(c.out["logprob"][live]).all(), name
            if name != "score" and name != "grad":
                assert torch.isnan(c.loss).all(), name
            if name.startswith("pairs"):
                assert torch.isnan(reward).all(), name
            if name in ("grad", "policy", "pairs"):
                assert torch.isnan(c.grad[live]).all() and (c.grad[~live] == 0).all(), name
                c.grad.fill_(-7.0)
            assert (c.gflat == -7).all(), name
    # another handle is not affected
    for name, call in calls(sampler, c):
        call()
        assert (c.status == 0).all() and torch.isfinite(c.out["logprob"]).all(), name
        assert name in ("score", "grad") or torch.isfinite(c.loss).all(), name


@pytest.mark.parametrize("bad", [[0, 3, 9, 5, 10], [0, 6, 9, 0, 4, 5, 7], [4, 10, 4, 10, 4, 10, 4, 10, 4], [9, 3, 0],
                                 [0, 8, 2, 6, 10], [0, 3, 5, 8, 11], [2, 5, -4, 7, 9]])
@pytest.mark.parametrize("kind,V,scale", [("f32", 301, 1), ("bf16", 301, 60)])
def test_answers_that_overlap(sampler, bad, kind, V, scale):
    """Offsets that decrease or leave the rows: defined rewards and gradients, the same bits each time, and nothing
    written beside the gradient. Offsets `scale` times as long have each answer's rows in several threads."""
    import torch

    c = Rows(15, 10 * scale, V, kind, kept=0.9, pad=3)
    offsets = np.array(bad, np.int32) * scale
    pairs = len(bad) // 2
    reward = torch.full((2 * pairs,), -7.0, device="cuda:0")
    call = lambda: sampler.preference_loss(  # noqa: E731
        seq_offsets=torch.from_numpy(offsets).cuda(), out_loss=c.loss, out_reward=reward, out_grad=c.grad, **c.kw())
    call()
    got = L.preference(c.x, c.tokens, offsets, None, c.T, c.weight)
    tol = c.check_rows(got, entropy=False)
    assert torch.isnan(c.loss).item()
    np.testing.assert_array_equal(np.isnan(reward.cpu().numpy()), np.isnan(got["reward"]))
    # as in test_preference_loss: the sigmoid has a slope of at most 1/4, in the margin's error
    w = c.weight.astype(np.float64)
    t_by = np.zeros(c.n)
    for i in range(pairs):
        if np.isnan(got["reward"][2 * i:2 * i + 2]).any():
            continue
        t_z = 0.0
        for s in (2 * i, 2 * i + 1):
            at = slice(offsets[s], offsets[s + 1])
            t_z += 0.1 * ((w * tol["logprob"])[at]).sum() + 3 * EPS * (abs(got["reward"][s]) + 1)
        for s in (2 * i, 2 * i + 1):
            at = slice(offsets[s], offsets[s + 1])
            t_by[at] = w[at] * 0.1 / pairs * (t_z / 4 + EPS)
    c.check_grad(got, tol, got["by_logprob"], t_by + 8 * EPS * np.abs(got["by_logprob"]))
    first = c.grad.clone(), reward.clone()
    for _ in range(20):
        c.grad.fill_(-7.0)
        call()
        for a, b in zip(first, (c.grad, reward)):
            assert torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                               b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))


@pytest.mark.parametrize("shape", [dict(n=9, V=7, kind="bf16", pad=1), dict(n=40, V=1000, kept=0.6, heat=True),
                                   dict(n=300, V=3001, kind="bf16", kept=0.7, shift=3), dict(n=60, V=16001, banned=0.3),
                                   dict(n=24, V=128000, kind="bf16", kept=0.8), dict(n=160, V=40961, kept=0.9, pad=1)],
                         ids=_id)
@pytest.mark.parametrize("mean", [False, True])
def test_preference_loss_without_the_gradient(sampler, shape, mean):
    """The outputs of the form with the gradient, bit for bit, and what the definition says."""
    import torch

    c = Rows(16, **shape)
    lp = L.score(c.x, c.tokens, c.T, c.weight)["logprob"]
    ref = (lp + 0.3 * c.rng.standard_normal(c.n)).astype(np.float32)
    offsets = np.array([0, c.n // 3, c.n // 2, c.n // 2, c.n], np.int32)
    reward = torch.full((4,), -7.0, device="cuda:0")
    kw = dict(beta=0.4, margin=0.25, label_smoothing=0.1, mean_over_tokens=mean)
    ins = dict(seq_offsets=torch.from_numpy(offsets).cuda(), ref_logprob=torch.from_numpy(ref).cuda(), out_loss=c.loss,
               out_reward=reward, **kw, **c.kw())
    sampler.preference_loss(out_grad=c.grad, **ins)
    first = [t.clone() for t in (c.loss, reward, c.out["logprob"], c.status)]
    for t in (c.loss, reward, c.out["logprob"]):
        t.fill_(-7.0)
    c.status.fill_(-7)
    c.gflat.fill_(-7.0)
    sampler.preference_loss(**ins)
    for a, b in zip(first, (c.loss, reward, c.out["logprob"], c.status)):
        assert torch.equal(a, b)
    assert (c.gflat == -7.0).all()
    got = L.preference(c.x, c.tokens, offsets, ref.astype(np.float64), c.T, c.weight, **kw)
    tol = c.check_rows(got, entropy=False)
    w = np.ones(c.n) if c.weight is None else c.weight.astype(np.float64)
    t_reward = np.zeros(4)
    for s in range(4):
        at = slice(offsets[s], offsets[s + 1])
        share = 1.0 / w[at].sum() if mean and w[at].sum() else 1.0
        t_reward[s] = 0.4 * share * ((w * tol["logprob"])[at]).sum() + 2 * EPS * abs(got["reward"][s])
    assert (np.abs(reward.double().cpu().numpy() - got["reward"]) <= t_reward).all()
    # beta, the margin and the smoothing are floats; the loss has a slope of at most 1 in a margin
    t_z = t_reward[0::2] + t_reward[1::2] + EPS * (np.abs(got["reward"]).max() + 1.25)
    assert abs(c.loss.item() - got["loss"]) <= t_z.sum() / 2 + 4 * EPS * (1 + abs(got["loss"]))
