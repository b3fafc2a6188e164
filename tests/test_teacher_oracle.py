"""The most likely tokens and distillation: the oracle against other forms and differences, and what the host refuses
(no GPU)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import oracle.teacher as O


def test_top_against_scipy():
    from scipy.special import log_softmax, logsumexp
    rng = np.random.default_rng(0)
    x = np.round(rng.standard_normal((6, 50)) * 4) / 2  # ties
    x[1, :20] = -np.inf
    x[2, 3:] = -np.inf
    T = np.linspace(0.5, 2, 6).astype(np.float32)
    got = O.top(x, 8, tokens=np.arange(6), temperature=T)
    for r in range(6):
        lp = log_softmax(x[r] / T[r])
        order = sorted(range(50), key=lambda v: (-x[r, v], v))[:8]
        order = [v for v in order if x[r, v] > -np.inf]
        assert list(got["ids"][r]) == order + [-1] * (8 - len(order))
        np.testing.assert_allclose(got["logprobs"][r, :len(order)], lp[order], rtol=1e-12, atol=1e-12)
        rest = [v for v in range(50) if v not in order]
        np.testing.assert_allclose(got["rest"][r], logsumexp(lp[rest]), rtol=1e-9, atol=1e-12)
        np.testing.assert_allclose(got["logprob"][r], lp[r], rtol=1e-12)


def _lists(rng, x, k, T=1.0):
    z = x + 0.7 * rng.standard_normal(x.shape)
    lp = z / T - np.log(np.exp(z / T).sum(1, keepdims=True))
    ids = np.argsort(-lp, 1)[:, :k].astype(np.int32)
    l = np.take_along_axis(lp, ids, 1)
    rest = np.log(1 - np.exp(l).sum(1))
    return ids, l.astype(np.float32), rest.astype(np.float32)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("coef", [0.0, 0.4])
def test_distill_gradient_against_differences(tail, coef):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 12))
    ids, l, rest = _lists(rng, x, 5)
    ids[2, 3:] = -1
    tok, T, w = np.array([0, 5, 7, 11]), np.array([1.0, 0.7, 1.3, 1.0], np.float32), np.array([0.5, 1.0, 2.0, 0.0])
    kw = dict(ids=ids, logprobs=l, rest=rest if tail else None, tokens=tok, token_coef=coef, temperature=T, weight=w)
    got = O.distill(x, **kw)
    for r in range(4):
        for v in range(12):
            d = np.zeros_like(x)
            d[r, v] = 1e-5
            n = (O.distill(x + d, **kw)["loss"] - O.distill(x - d, **kw)["loss"]) / 2e-5
            np.testing.assert_allclose(got["grad"][r, v], n, rtol=1e-6, atol=1e-9)


def test_distill_of_the_teacher_itself_is_0():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 40)) * 3
    t = O.top(x, 7)
    got = O.distill(x, t["ids"], t["logprobs"], t["rest"])
    np.testing.assert_allclose(got["kl"], 0, atol=1e-12)
    np.testing.assert_allclose(got["grad"], 0, atol=1e-12)


def test_distill_over_the_whole_vocabulary_is_the_divergence():
    from scipy.special import log_softmax
    rng = np.random.default_rng(3)
    x, z = rng.standard_normal((2, 3, 9))
    lt = log_softmax(z, 1)
    got = O.distill(x, np.tile(np.arange(9, dtype=np.int32), (3, 1)), lt, np.full(3, -np.inf))
    np.testing.assert_allclose(got["kl"], (np.exp(lt) * (lt - log_softmax(x, 1))).sum(1), rtol=1e-12)
    np.testing.assert_allclose(got["grad"], np.exp(log_softmax(x, 1)) - np.exp(lt), atol=1e-12)


# ------------------------------------------------------------------ what the host refuses
@pytest.fixture(scope="module")
def handle():
    """A handle's memory without a device: the host's checks read its limits and come before any CUDA call. (Its losses
    take no rows: the workspace is not there.)"""
    import decode_step_token_gb300 as d
    from decode_step_token_gb300 import build
    build.build_library()
    d.load_library()

    class Limits(ctypes.Structure):
        _fields_ = [("device", ctypes.c_int), ("num_sms", ctypes.c_int), ("max_rows", ctypes.c_int64),
                    ("max_vocab", ctypes.c_int64), ("rest", ctypes.c_char * 4096)]

    h = Limits(0, 152, 64, 1000)
    return ctypes.addressof(h), h


def _rows(**kw):
    import decode_step_token_gb300 as d
    a = dict(logits=4096, dtype=d.SAMPLER_DTYPE_F32, n_rows=4, vocab=100, row_stride=100, tokens=4096)
    a.update(kw)
    return d.sampler_rows_t(**a)


@pytest.mark.parametrize("rows,top,code", [
    (dict(), dict(top_n=0), -9), (dict(), dict(top_n=129), -9), (dict(), dict(top_n=-1), -9),
    (dict(), dict(out_top_ids=None), -1), (dict(), dict(out_top_logprobs=None), -1), (dict(out_grad=4096, grad_stride=100), dict(), -8),
    (dict(tokens=None, out_logprob=4096), dict(), -1), (dict(logits=None), dict(), -1), (dict(vocab=0), dict(), -2),
    (dict(row_stride=99), dict(), -2), (dict(n_rows=65), dict(), -3), (dict(vocab=1001, row_stride=1001), dict(), -3),
    (dict(dtype=3), dict(), -4), (dict(), dict(out_top_ids=4097), -2), (dict(), dict(out_rest_logprob=4098), -2),
    (dict(out_entropy=4097), dict(), -2), (dict(n_rows=0), dict(), 0), (dict(n_rows=0, tokens=None), dict(top_n=0), -9)])
def test_top_refusals(handle, rows, top, code):
    import decode_step_token_gb300 as d
    t = d.sampler_top_t(**{**dict(top_n=5, out_top_ids=4096, out_top_logprobs=4096), **top})
    assert d.sampler_score_top(handle[0], _rows(**rows), t, 0) == code


@pytest.mark.parametrize("rows,kw,code", [
    (dict(n_rows=1), dict(), -3),  # above the (missing) workspace's rows
    (dict(n_rows=0), dict(out_loss=None), -1), (dict(n_rows=0, out_entropy=4096), dict(), -8),
    (dict(n_rows=0), dict(top_n=0), -9), (dict(n_rows=0), dict(top_n=129), -9), (dict(n_rows=0), dict(token_coef=-0.1), -9),
    (dict(n_rows=0), dict(token_coef=float("nan")), -9), (dict(n_rows=0), dict(token_coef=float("inf")), -9),
    (dict(n_rows=0), dict(grad_scale=float("inf")), -9), (dict(n_rows=0), dict(out_loss=4097), -2),
    (dict(n_rows=0), dict(teacher_ids=4098), -2), (dict(n_rows=0), dict(teacher_rest=4097), -2),
    (dict(n_rows=0), dict(out_kl=4099), -2), (dict(n_rows=0), dict(grad_scale_dev=4099), -2), (dict(vocab=0), dict(), -2),
    (dict(tokens=None, out_logprob=4096), dict(), -1), (dict(out_grad=4096, grad_stride=99), dict(), -2),
    (dict(out_grad=4096, grad_stride=104), dict(), -2)])
def test_distill_refusals(handle, rows, kw, code):
    import decode_step_token_gb300 as d
    q = d.sampler_distill_t(**{**dict(top_n=5, teacher_ids=4096, teacher_logprobs=4096, grad_scale=1.0, out_loss=4096), **kw})
    assert d.sampler_distill_loss(handle[0], _rows(**rows), q, 0) == code


def test_null_arguments(handle):
    import decode_step_token_gb300 as d
    lib, none = d.load_library(), None
    assert d.sampler_score_top(none, _rows(), d.sampler_top_t(top_n=5), 0) == -1
    assert d.sampler_distill_loss(none, _rows(), d.sampler_distill_t(top_n=5), 0) == -1
    assert lib.sampler_score_top(handle[0], ctypes.byref(_rows()), None, None) == -1
    assert lib.sampler_distill_loss(handle[0], ctypes.byref(_rows(n_rows=0)), None, None) == -1
    assert lib.sampler_score_top(handle[0], None, None, None) == -1


def test_struct_layouts(tmp_path):
    import decode_step_token_gb300 as d
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    body, want = ["#include <stdio.h>", "#include <stddef.h>", '#include "sampler.h"', "int main(void){"], []
    for name in ("sampler_top_t", "sampler_distill_t"):
        st = getattr(d, name)
        body.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(st))
        for f in st._fields_:
            body.append(f'printf("%zu\\n", offsetof({name}, {f[0]}));')
            want.append(getattr(st, f[0]).offset)
    body.append('printf("%d\\n", SAMPLER_MAX_ALTERNATIVES);return 0;}')
    want.append(d.SAMPLER_MAX_ALTERNATIVES)
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(body))
    subprocess.run(["gcc", f"-I{root}/include", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert [int(x) for x in out.split()] == want
