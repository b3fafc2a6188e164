"""The C ABI library builds, loads and exports what include/sampler.h declares (no GPU)."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sampler.h")


@pytest.fixture(scope="module")
def lib():
    from decode_step_token_gb300 import build
    build.build_library()
    import decode_step_token_gb300 as d
    return d.load_library()


def declared_functions():
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(sampler_[a-z_]+)\s*\(", text)))


def test_header_declares_the_documented_entry_points():
    names = declared_functions()
    for n in ("sampler_create", "sampler_sample", "sampler_destroy", "sampler_status_string"):
        assert n in names


def test_library_exports_every_declared_symbol(lib):
    for name in declared_functions():
        assert hasattr(lib, name), name
    out = subprocess.run(["nm", "-D", "--defined-only", lib._name], capture_output=True, text=True)
    exported = set(re.findall(r"\bT (sampler_\w+)", out.stdout))
    assert set(declared_functions()) <= exported


def test_python_binding_uses_the_abi_names(lib):
    import decode_step_token_gb300 as d
    assert set(d.EXPORTED) == set(declared_functions())


def test_struct_layouts_match_the_header(tmp_path):
    import decode_step_token_gb300 as d
    structs = [("sampler_args_t", d.sampler_args_t), ("sampler_config_t", d.sampler_config_t),
               ("sampler_ext_t", d.sampler_ext_t), ("sampler_lm_head_t", d.sampler_lm_head_t)]
    src = tmp_path / "layout.c"
    body = ['#include <stdio.h>', '#include <stddef.h>', '#include "sampler.h"', "int main(void){"]
    for name, st in structs:
        body.append(f'printf("%zu\\n", sizeof({name}));')
        for f in st._fields_:
            body.append(f'printf("%zu\\n", offsetof({name}, {f[0]}));')
    body.append("return 0;}")
    src.write_text("\n".join(body))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", f"-I{os.path.dirname(HEADER)}", str(src), "-o", str(exe)], check=True)
    vals = iter(int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                               check=True).stdout.split())
    for name, st in structs:
        assert next(vals) == ctypes.sizeof(st), name
        for f in st._fields_:
            assert getattr(st, f[0]).offset == next(vals), (name, f[0])


def test_host_checks_without_a_gpu(lib):
    import decode_step_token_gb300 as d
    assert d.sampler_abi_version() >> 16 == 1
    assert "limits" in d.sampler_status_string(-3)
    # NULL handle / NULL config are rejected before any CUDA call
    rc, h = d.sampler_create(d.sampler_config_t(0, 0, 10, 0, 0))
    assert rc == d._binding.SAMPLER_ERR_BAD_SHAPE and not h.value
    assert lib.sampler_sample(None, None, None) == d._binding.SAMPLER_ERR_NULL_ARG
    d.sampler_destroy(None)


def test_product_path_does_not_touch_the_oracle():
    pkg = os.path.join(ROOT, "decode_step_token_gb300")
    for dirpath, _, files in os.walk(pkg):
        for f in files:
            if f.endswith((".py", ".cu", ".cuh", ".h", ".cpp")):
                text = open(os.path.join(dirpath, f)).read()
                assert "oracle" not in text.lower().replace("oracle-free", ""), f


def test_struct_layouts_of_scoring_and_the_8bit_head(tmp_path):
    import decode_step_token_gb300 as d
    structs = [(name, getattr(d, name)) for name in ("sampler_rows_t", "sampler_policy_t", "sampler_preference_t",
                                                     "sampler_quantize_t", "sampler_scaled_head_t")]
    body = ["#include <stdio.h>", "#include <stddef.h>", '#include "sampler.h"', "int main(void){"]
    want = []
    for name, st in structs:
        body.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(st))
        for f in st._fields_:
            body.append(f'printf("%zu\\n", offsetof({name}, {f[0]}));')
            want.append(getattr(st, f[0]).offset)
    body.append('printf("%d\\n%d\\n", SAMPLER_LOSS_MAX_ROWS, SAMPLER_ERR_BAD_VALUE);return 0;}')
    want += [d.SAMPLER_LOSS_MAX_ROWS, d.SAMPLER_ERR_BAD_VALUE]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(body))
    subprocess.run(["gcc", f"-I{os.path.dirname(HEADER)}", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert [int(x) for x in out.split()] == want


def test_host_checks_of_scoring_and_the_8bit_head_without_a_gpu(lib):
    """A NULL handle or argument is refused before any CUDA call."""
    import decode_step_token_gb300 as d
    b = d._binding
    rows, none = d.sampler_rows_t(), None
    assert b.sampler_score(none, rows, 0) == b.SAMPLER_ERR_NULL_ARG
    assert b.sampler_score_grad(none, rows, 0, 0, 0) == b.SAMPLER_ERR_NULL_ARG
    assert b.sampler_policy_loss(none, rows, d.sampler_policy_t(), 0) == b.SAMPLER_ERR_NULL_ARG
    assert b.sampler_preference_loss(none, rows, d.sampler_preference_t(), 0) == b.SAMPLER_ERR_NULL_ARG
    assert b.sampler_quantize_blocks(none, d.sampler_quantize_t(), 0) == b.SAMPLER_ERR_NULL_ARG
    assert b.sampler_lm_head_scaled(none, d.sampler_scaled_head_t(), 0, 0, 1, 1, 1, 0) == b.SAMPLER_ERR_NULL_ARG
    assert (b.sampler_lm_head_scaled_sample(none, d.sampler_scaled_head_t(), d.sampler_args_t(), none, 0)
            == b.SAMPLER_ERR_NULL_ARG)
