"""The double-precision definitions of scoring, the losses and the 8-bit LM head
(oracle/losses.py) against torch's autograd, central differences, torch's own
e4m3 rounding and scipy; and the refusals that need no GPU. CPU only."""
import ctypes

import numpy as np
import pytest
import torch
from scipy.special import log_softmax

import oracle.losses as L


def _case(seed, n=7, V=23, banned=False):
    rng = np.random.default_rng(seed)
    x = 2.0 * rng.standard_normal((n, V))
    tokens = rng.integers(0, V, n).astype(np.int32)
    if banned:
        x[rng.random((n, V)) < 0.3] = -np.inf
        x[np.arange(n), tokens] = 1.0
    T = rng.uniform(0.5, 1.5, n).astype(np.float32)
    w = rng.uniform(0.2, 1.0, n).astype(np.float32)
    w[n // 2] = 0.0
    return rng, x, tokens, T, w


def test_score_is_the_log_softmax():
    _, x, tokens, T, w = _case(0, banned=True)
    got = L.score(x, tokens, T, w)
    want = log_softmax(x / T.astype(np.float64)[:, None], axis=1)
    live = w != 0
    np.testing.assert_allclose(got["logprob"][live], want[np.arange(7), tokens][live], rtol=1e-13)
    p = np.exp(want)
    h = -np.where(p > 0, p * np.where(p > 0, want, 0.0), 0.0).sum(1)
    np.testing.assert_allclose(got["entropy"][live], h[live], rtol=1e-13)
    assert got["logprob"][~live] == 0 and got["entropy"][~live] == 0


def test_score_of_rows_of_the_lowest_value():
    x = np.full((1, 8), -np.finfo(np.float32).max, np.float64)
    got = L.score(x, np.zeros(1, np.int32))
    assert got["logprob"][0] == -np.log(8) and abs(got["entropy"][0] - np.log(8)) < 1e-15


def _differences(f, x, grad):
    """Central differences of f at every finite entry of x against grad."""
    h = 1e-6
    for r in range(x.shape[0]):
        for v in range(x.shape[1]):
            if not np.isfinite(x[r, v]):
                assert grad[r, v] == 0
                continue
            a, b = x.copy(), x.copy()
            a[r, v] += h
            b[r, v] -= h
            # truncation h^2 f''' and cancellation 1e-16 |f| / h are both below 1e-9 here
            assert abs((f(a) - f(b)) / (2 * h) - grad[r, v]) < 2e-9 * max(1.0, abs(f(x))), (r, v)


@pytest.mark.parametrize("seed,banned", [(1, False), (2, True)])
def test_policy_gradient(seed, banned):
    rng, x, tokens, T, w = _case(seed, banned=banned)
    lp = L.score(x, tokens, T)["logprob"]
    # ratios on both sides of both clips, none within the differences' step of one
    old = lp - np.log([0.5, 0.75, 0.9, 1.0, 1.1, 1.4, 2.0])
    adv = rng.permutation([-1.5, -1.0, -0.5, 0.0, 0.5, 1.0, 1.5])
    ref = lp + rng.normal(0, 0.5, 7)
    kw = dict(old=old, advantage=adv, ref=ref, temperature=T, weight=w, clip_low=0.2, clip_high=0.3, kl_coef=0.1,
              entropy_coef=0.05)
    got = L.policy(x, tokens, **kw)
    _differences(lambda y: L.policy(y, tokens, **kw)["loss"], x, got["grad"])
    t = torch.tensor(x, requires_grad=True)
    logp = torch.log_softmax(t / torch.tensor(T).double()[:, None], 1)
    tlp = logp[torch.arange(7), torch.tensor(tokens).long()]
    ratio = torch.exp(tlp - torch.tensor(old))
    A = torch.tensor(adv)
    d = torch.tensor(ref) - tlp
    inside = torch.where(logp > -np.inf, logp, torch.zeros(()).double())
    each = (-torch.minimum(ratio * A, ratio.clamp(0.8, 1.3) * A) + 0.1 * (torch.exp(d) - d - 1)
            + 0.05 * (torch.exp(logp) * inside).sum(1))
    loss = (each * torch.tensor(w).double())[torch.tensor(w) != 0].sum()
    loss.backward()
    assert abs(loss.item() - got["loss"]) < 1e-12
    if not banned:
        np.testing.assert_allclose(got["grad"], t.grad.numpy(), rtol=1e-10, atol=1e-13)


@pytest.mark.parametrize("mean", [False, True])
def test_preference_gradient(mean):
    rng, x, tokens, T, w = _case(3, n=11)
    offsets = np.array([0, 3, 5, 5, 9], np.int32)  # an empty answer; the last rows are in none
    ref = rng.normal(-3, 1, 11)
    kw = dict(offsets=offsets, ref=ref, temperature=T, weight=w, beta=0.7, margin=0.1, label_smoothing=0.1,
              mean_over_tokens=mean)
    got = L.preference(x, tokens, **kw)
    assert (got["grad"][9:] == 0).all() and got["reward"][2] == 0
    _differences(lambda y: L.preference(y, tokens, **kw)["loss"], x, got["grad"])
    z = got["reward"][0::2] - got["reward"][1::2] - 0.1
    sure = torch.nn.functional.logsigmoid
    zt = torch.tensor(z)
    assert abs((-0.9 * sure(zt) - 0.1 * sure(-zt)).mean().item() - got["loss"]) < 1e-13


def test_score_gradient():
    rng, x, tokens, T, w = _case(4)
    a, b = rng.standard_normal(7), rng.standard_normal(7)

    def f(y):
        s = L.score(y, tokens, T, w)
        return float((a * s["logprob"] + b * s["entropy"]).sum())

    _differences(f, x, L.logits_grad(L.score(x, tokens, T, w), tokens, a, b, T, w))


def test_status_rows():
    x = np.zeros((6, 5))
    x[0, 1], x[1, 2], x[2] = np.nan, np.inf, -np.inf
    got = L.score(x, np.array([0, 0, 0, 5, 0, 0]), np.array([1, 1, 1, 1, -1, 1e-6], np.float32))
    np.testing.assert_array_equal(got["status"], [1, 1, 2, 3, 3, 0])
    assert abs(got["logprob"][5] + np.log(5)) < 1e-15  # T below 1e-5 reads as 1


def test_e4m3_codes_match_torch():
    rng = np.random.default_rng(5)
    t = L.e4m3_table()
    ours = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(t, ours)
    p = t[:127]
    x = np.concatenate([p, (p[1:] + p[:-1]) / 2, rng.uniform(0, 448, 20000), 2.0 ** rng.uniform(-12, 8.8, 20000)])
    x = np.concatenate([x, -x]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(L.to_e4m3(x.astype(np.float64)), want)


def test_quantize_reaches_the_largest_value():
    rng = np.random.default_rng(6)
    x = rng.standard_normal((200, 300)).astype(np.float32)
    x[130:, :128] = 0
    x[3, 200] = np.nan
    for rows in (1, 128):
        codes, scales = L.quantize(x, rows)
        back = L.e4m3_table()[codes] * np.repeat(np.repeat(scales, rows, 0)[:200], 128, 1)[:, :300]
        fine = np.isfinite(back)
        assert np.isnan(back[3, 128:256]).all() and fine.sum() == (60000 - 128 * (1 if rows == 1 else 128))
        # half a step of 4 bits, with the scale's own rounding (three operations)
        lim = np.abs(x) * 2.0 ** -4 + np.repeat(np.repeat(scales, rows, 0)[:200], 128, 1)[:, :300] * 2.0 ** -10
        assert (np.abs(back - x)[fine] <= (lim * (1 + 2.0 ** -20))[fine]).all()


def test_scaled_head_is_the_dequantised_product():
    rng = np.random.default_rng(7)
    h, w = (rng.integers(0, 127, s).astype(np.uint8) for s in ((3, 200), (150, 200)))
    sh, sw = rng.uniform(0.1, 1, (3, 2)).astype(np.float32), rng.uniform(0.1, 1, (2, 2)).astype(np.float32)
    t = L.e4m3_table()
    H = t[h] * np.repeat(sh, 128, 1)[:, :200]
    W = t[w] * np.repeat(np.repeat(sw, 128, 0)[:150], 128, 1)[:, :200]
    np.testing.assert_allclose(L.scaled_head(h, sh, w, sw)[0], H @ W.T, rtol=1e-12)


# ------------------------------------------------------------------ what needs no GPU of the library
@pytest.fixture(scope="module")
def lib():
    from decode_step_token_gb300 import build
    build.build_library()
    import decode_step_token_gb300 as d
    return d.load_library()


def test_null_handles_are_refused(lib):
    import decode_step_token_gb300 as d
    null = d._binding.SAMPLER_ERR_NULL_ARG
    assert d.sampler_score(None, d.sampler_rows_t(), 0) == null
    assert d.sampler_score_grad(None, d.sampler_rows_t(), None, None, 0) == null
    assert d.sampler_policy_loss(None, d.sampler_rows_t(), d.sampler_policy_t(), 0) == null
    assert d.sampler_preference_loss(None, d.sampler_rows_t(), d.sampler_preference_t(), 0) == null
    assert d.sampler_quantize_blocks(None, d.sampler_quantize_t(), 0) == null
    assert d.sampler_lm_head_scaled(None, d.sampler_scaled_head_t(), 0, 1, 1, 1, 1, 0) == null
    assert lib.sampler_lm_head_scaled_sample(None, None, None, None, None) == null
    assert "range" in d.sampler_status_string(d.SAMPLER_ERR_BAD_VALUE)


def test_struct_layouts(tmp_path):
    import os
    import subprocess

    import decode_step_token_gb300 as d
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    names = ("sampler_rows_t", "sampler_policy_t", "sampler_preference_t", "sampler_quantize_t",
             "sampler_scaled_head_t")
    body = ['#include <stdio.h>', '#include <stddef.h>', '#include "sampler.h"', "int main(void){"]
    want = []
    for name in names:
        st = getattr(d, name)
        body.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(st))
        for f in st._fields_:
            body.append(f'printf("%zu\\n", offsetof({name}, {f[0]}));')
            want.append(getattr(st, f[0]).offset)
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(body + ["return 0;}"]))
    subprocess.run(["gcc", f"-I{include}", str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == want


def test_binding_refuses_what_it_can_see(lib):
    """Types, shapes and devices are checked before any address reaches the library."""
    import decode_step_token_gb300 as d
    s = object.__new__(d.Sampler)
    s._h, s.device = None, 0
    x = torch.zeros((4, 10))
    tok = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="is on cpu"):
        s.score(logits=x, tokens=tok)
    with pytest.raises(TypeError, match="logits"):
        s.score(logits=x.half(), tokens=tok)
    with pytest.raises(ValueError, match="contiguous rows"):
        s.score(logits=x.t(), tokens=tok)
    with pytest.raises(TypeError, match="src"):
        s.quantize_blocks(src=x.half(), out_values=x, out_scales=x)
    with pytest.raises(TypeError, match="hidden"):
        s.lm_head_scaled(hidden=x, hidden_scale=x, weight=x, weight_scale=x, logits=x)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_binding_refuses_rows_that_overlap(dtype):
    """A row stride below the width (a broadcast row, a sliding window) is no matrix: its rows do not lie where
    cols * row would put them."""
    from decode_step_token_gb300 import _matrix

    x = torch.zeros(64, dtype=dtype)
    for t in (x[:8].expand(5, 8), x.as_strided((5, 8), (3, 1)), x.as_strided((2, 8), (7, 1))):
        with pytest.raises(ValueError):
            _matrix("x", t, (dtype,), -1)
    assert _matrix("x", x[:8].expand(1, 8), (dtype,), -1) == (1, 8, 8)
    assert _matrix("x", x.as_strided((5, 8), (9, 1)), (dtype,), -1) == (5, 8, 9)
    assert _matrix("x", x.as_strided((1, 8), (0, 1)), (dtype,), -1) == (1, 8, 8)
    assert _matrix("x", x.view(8, 8)[:0], (dtype,), -1)[:2] == (0, 8)


def test_preference_rows_in_several_answers():
    """Offsets that decrease: the answer with its end before its begin and its pair are NaN, and so is the gradient of
    rows in more than one answer; the other rows keep theirs."""
    rng = np.random.default_rng(8)
    x, tok = rng.standard_normal((10, 30)), rng.integers(0, 30, 10)
    got = L.preference(x, tok, [0, 6, 9, 0, 4, 5, 7])
    # answers [0, 6) [6, 9) | [9, 0) [0, 4) | [4, 5) [5, 7)
    assert np.isnan(got["reward"]).tolist() == [False, False, True, False, False, False] and np.isnan(got["loss"])
    nan = np.isnan(got["grad"]).all(1)
    assert nan.tolist() == [True] * 7 + [False] * 3 and np.isfinite(got["grad"][~nan]).all()
    alone = L.preference(x, tok, [0, 6, 9])
    np.testing.assert_allclose(got["grad"][7:9], alone["grad"][7:9] / 3, rtol=1e-14)
    assert (got["grad"][9] == 0).all()
