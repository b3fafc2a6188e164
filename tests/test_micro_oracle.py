"""Microscaled 4 bits: the oracle against brute force, and what the host refuses (no GPU)."""
import ctypes
import itertools

import numpy as np
import pytest

import oracle.micro as M

E4M3 = np.array([M.e4m3_value(c) for c in range(127)])


def test_e4m3_codes_round_trip():
    for c, v in enumerate(E4M3):
        assert M.e4m3_code(v) == c
    assert E4M3[126] == 448.0 and E4M3[1] == 2.0 ** -9 and E4M3[8] == 2.0 ** -6


def _nearest_of(x, table):
    """Index of the nearest table entry; of two as near, the even one."""
    d = np.abs(table - x)
    best = np.flatnonzero(d == d.min())
    return int(best[0] if len(best) == 1 else best[best % 2 == 0][0])


@pytest.mark.parametrize("block", [16, 32])
def test_quantize_against_every_code(block):
    rng = np.random.default_rng(block)
    rows, cols = 7, 70
    # few digits, so that many quotients lie halfway between two codes
    x = rng.integers(-40, 41, (rows, cols)) * 2.0 ** rng.integers(-3, 3, (rows, 1))
    x[3] = 0
    x[4, 5:60] *= 1e-3
    x = x.astype(np.float32)
    packed, scales, row_scale, values = M.quantize(x, block)
    place, size = M.scale_place(rows, cols, block)
    assert size == len(scales) and len(set(place.ravel())) == place.size
    for r, b in itertools.product(range(rows), range(-(-cols // block))):
        v = x[r, b * block:(b + 1) * block].astype(np.float64)
        m = np.abs(v).max()
        if block == 16:
            M_ = max(np.abs(x[r]).max(), M.LEAST)
            g = row_scale[r]
            assert M_ <= 2688 * float(g) and not M_ <= 1344 * float(g) and np.log2(g) % 1 == 0
            code = _nearest_of(m / 6 / float(g), E4M3)
            s = E4M3[code] * float(g)
        else:
            code = int(scales[place[r, b]])
            s = 2.0 ** (code - 127)
            assert m <= 6 * s and (code == 0 or m > 3 * s)
        assert scales[place[r, b]] == code
        for i, y in enumerate(v):
            k = _nearest_of(min(abs(y) / s, 6.0), M.CODES) if s else 0
            col = b * block + i
            got = packed[r, col // 2] >> 4 * (col % 2) & 15
            assert got & 7 == k, (r, col, y, s)
            assert values[r, col] == np.copysign(M.CODES[k], y) * s
    np.testing.assert_array_equal(M.values(packed, scales, row_scale, cols, block), values)


@pytest.mark.parametrize("block", [16, 32])
def test_quantize_what_is_not_finite(block):
    x = np.ones((2, 96), np.float32)
    x[0, 40], x[1, 3] = np.nan, -np.inf
    packed, scales, row_scale, values = M.quantize(x, block)
    bad = np.zeros((2, 96), bool)
    bad[0, 40 // block * block:40 // block * block + block] = True
    bad[1, :block] = True
    assert (np.isnan(values) == bad).all() and np.isfinite(row_scale).all()
    again = M.values(packed, scales, row_scale, 96, block)
    assert (np.isnan(again) == bad).all()
    np.testing.assert_allclose(values[~bad], 1.0, rtol=2.0 ** -4)


@pytest.mark.parametrize("block", [16, 32])
def test_small_and_large_rows(block):
    x = np.array([[1e-38, -3e-39, 0.0], [3.4e38, -1e38, 1.0], [1e-30, 5e-31, -2e-31]], np.float32)
    packed, scales, row_scale, values = M.quantize(x, block)
    assert np.isfinite(values).all()
    np.testing.assert_allclose(values[1, :2], x[1, :2], rtol=0.25)
    if block == 32:
        np.testing.assert_allclose(values[0, :2], x[0, :2].astype(float), rtol=0.5)
        np.testing.assert_allclose(values[2], x[2], rtol=0.25)


# ------------------------------------------------------------------ what the host refuses
@pytest.fixture(scope="module")
def handle():
    """A handle's memory without a device: the host's checks read its limits and come before any CUDA call."""
    import decode_step_token_gb300 as d
    from decode_step_token_gb300 import build
    build.build_library()
    d.load_library()

    class Limits(ctypes.Structure):
        _fields_ = [("device", ctypes.c_int), ("num_sms", ctypes.c_int), ("max_rows", ctypes.c_int64),
                    ("max_vocab", ctypes.c_int64), ("rest", ctypes.c_char * 4096)]

    h = Limits(0, 152, 64, 1000)
    return ctypes.addressof(h), h


def _quantize(**kw):
    import decode_step_token_gb300 as d
    a = dict(src=4096, dtype=d.SAMPLER_DTYPE_BF16, rows=4, cols=33, src_stride=33, block=16, values=4096, values_stride=17,
             scales=4096, row_scale=4096)
    a.update(kw)
    return d.sampler_micro_t(*[a[f] for f, _ in d.sampler_micro_t._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(block=8), -9), (dict(block=64), -9), (dict(rows=-1), -2), (dict(cols=0), -2), (dict(cols=(1 << 24) + 1), -2),
    (dict(src_stride=32), -2), (dict(values_stride=16), -2), (dict(dtype=7), -4), (dict(src=None), -1),
    (dict(values=None), -1), (dict(scales=None), -1), (dict(row_scale=None), -1), (dict(src=4097), -2),
    (dict(scales=4104), -2), (dict(row_scale=4098), -2), (dict(rows=0), 0)])
def test_quantize_refusals(handle, kw, code):
    import decode_step_token_gb300 as d
    assert d.sampler_quantize_micro(handle[0], _quantize(**kw), 0) == code


def _rows(**kw):
    import decode_step_token_gb300 as d
    a = dict(values=4096, values_stride=17, scales=4096, row_scale=None, rows=4, cols=33, block=16, ids=None, n=4, out=4096,
             dtype=d.SAMPLER_DTYPE_F32, out_stride=33)
    a.update(kw)
    return d.sampler_micro_rows_t(*[a[f] for f, _ in d.sampler_micro_rows_t._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(block=0), -9), (dict(n=5), -2), (dict(n=-1), -2), (dict(n=1 << 31, ids=4096), -2), (dict(out_stride=32), -2),
    (dict(values_stride=16), -2), (dict(cols=0), -2), (dict(dtype=-1), -4), (dict(out=None), -1), (dict(values=None), -1),
    (dict(scales=None), -1), (dict(out=4098), -2), (dict(ids=4097), -2), (dict(scales=4100), -2),
    (dict(row_scale=4099), -2), (dict(n=0), 0)])
def test_rows_refusals(handle, kw, code):
    import decode_step_token_gb300 as d
    assert d.sampler_micro_rows(handle[0], _rows(**kw), 0) == code


def _head(**kw):
    import decode_step_token_gb300 as d
    a = dict(hidden=4096, hidden_scale=4096, hidden_row_scale=None, weight=4096, weight_scale=4096, weight_row_scale=None,
             hidden_dim=100, hidden_stride=64, weight_stride=64, block=16)
    a.update(kw)
    return d.sampler_micro_head_t(*[a[f] for f, _ in d.sampler_micro_head_t._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(block=128), -9), (dict(hidden_dim=0), -2), (dict(hidden_dim=129), -2), (dict(hidden_dim=(1 << 24) + 1), -2),
    (dict(hidden_stride=56), -2), (dict(weight_stride=48), -2), (dict(hidden=4104), -2), (dict(weight=4097), -2),
    (dict(hidden_scale=4100), -2), (dict(weight_scale=4104), -2), (dict(hidden_row_scale=4097), -2),
    (dict(weight_row_scale=4098), -2), (dict(hidden=None), -1), (dict(weight=None), -1), (dict(hidden_scale=None), -1),
    (dict(weight_scale=None), -1)])
def test_head_refusals(handle, kw, code):
    import decode_step_token_gb300 as d
    lm = _head(**kw)
    assert d.sampler_lm_head_micro(handle[0], lm, 4096, d.SAMPLER_DTYPE_F32, 200, 4, 200, 0) == code
    args = d.sampler_args_t(logits=4096, dtype=d.SAMPLER_DTYPE_F32, n_rows=4, vocab=200, row_stride=200, temperature=4096,
                            out_tokens=4096)
    assert d.sampler_lm_head_micro_sample(handle[0], lm, args, None, 0) == code


def test_head_refusals_of_the_logits(handle):
    import decode_step_token_gb300 as d
    f32, bf16, h = d.SAMPLER_DTYPE_F32, d.SAMPLER_DTYPE_BF16, handle[0]
    call = lambda *a: d.sampler_lm_head_micro(h, _head(), *a)  # noqa: E731
    assert call(4096, 5, 200, 4, 200, 0) == -4
    assert call(4096, f32, 199, 4, 200, 0) == -2
    assert call(4096, f32, 200, -1, 200, 0) == -2
    assert call(4098, f32, 200, 4, 200, 0) == -2
    assert call(4097, bf16, 200, 4, 200, 0) == -2
    assert call(4096, f32, 2000, 4, 1001, 0) == -3
    assert call(4096, f32, 200, 1 << 31, 200, 0) == -3
    assert call(0, f32, 200, 4, 200, 0) == -1
    assert call(0, f32, 200, 0, 200, 0) == 0
    for entry in (lambda: d.sampler_quantize_micro(None, _quantize(), 0), lambda: d.sampler_micro_rows(None, _rows(), 0),
                  lambda: d.sampler_lm_head_micro(None, _head(), 4096, f32, 200, 4, 200, 0)):
        assert entry() == -1


def test_scale_bytes(handle):
    import decode_step_token_gb300 as d
    for rows, cols, block in [(1, 1, 16), (128, 64, 16), (129, 65, 16), (300, 1000, 32), (0, 5, 32)]:
        assert d.sampler_micro_scale_bytes(rows, cols, block) == M.scale_place(max(rows, 0), cols, block)[1]
    for rows, cols, block in [(1, 0, 16), (-1, 5, 16), (1, 5, 24), (1, (1 << 24) + 1, 16)]:
        assert d.sampler_micro_scale_bytes(rows, cols, block) == -1


def test_struct_layouts(tmp_path):
    import os
    import subprocess

    import decode_step_token_gb300 as d
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    body, want = ["#include <stdio.h>", "#include <stddef.h>", '#include "sampler.h"', "int main(void){"], []
    for name in ("sampler_micro_t", "sampler_micro_rows_t", "sampler_micro_head_t"):
        st = getattr(d, name)
        body.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(st))
        for f in st._fields_:
            body.append(f'printf("%zu\\n", offsetof({name}, {f[0]}));')
            want.append(getattr(st, f[0]).offset)
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(body + ["return 0;}"]))
    subprocess.run(["gcc", f"-I{root}/include", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert [int(x) for x in out.split()] == want
