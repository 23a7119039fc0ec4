"""The W8A8 layer's native module: what needs it, what does not, and when it is built anew."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "bit_w4a4_quantized_token_b200"


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_w4a4_quantized_token_b200 import build

    build.build()


def copy_without_module(where):
    """The package as built, but for the native module."""
    shutil.copytree(os.path.join(ROOT, PACKAGE), os.path.join(where, PACKAGE),
                    ignore=shutil.ignore_patterns("_w8a8_front*", "csrc", "__pycache__"))


def python(code, where):
    return subprocess.run([sys.executable, "-c", code], cwd=where, capture_output=True, text=True, timeout=300,
                          env=dict(os.environ, PYTHONPATH=str(where)))


WITHOUT = """
import torch
from bit_w4a4_quantized_token_b200 import layer
assert callable(layer.svdq_linear) and callable(layer.pack_weight)
packed = layer.PackedWeightW8A8(8, 32, torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8), None, None)
x = torch.zeros(4, 32, dtype=torch.bfloat16)
q = layer.QuantizedActW8A8(8, packed.w_codes, packed.w_scales)
for call in (lambda: layer.pack_weight_w8a8(torch.zeros(8, 32)), lambda: layer.quantize_act_w8a8(x, packed),
             lambda: layer.rms_norm_quantize_w8a8(x, None, None, packed), lambda: layer.gemm_w8a8(q, packed),
             lambda: layer.w8a8_linear(x, packed)):
    try:
        call()
    except ImportError as e:
        assert "not built" in str(e), e
    else:
        raise AssertionError("a W8A8 function ran without its native module")
print("as it should be")
"""


def test_the_4_bit_layer_does_not_need_the_module(tmp_path):
    """Without it the package imports, and the W8A8 functions say what is missing when they are called."""
    copy_without_module(tmp_path)
    r = python(WITHOUT, tmp_path)
    assert r.returncode == 0 and "as it should be" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("lacking", [None, "torch", "a torch with CUDA", "Python's headers"])
def test_the_library_is_built_without_what_the_module_needs(monkeypatch, capsys, tmp_path, lacking):
    """The library comes first, whatever the machine lacks for the module, and what is not built is said."""
    import sysconfig

    from bit_w4a4_quantized_token_b200 import build

    outputs = []
    monkeypatch.setattr(build, "_compile", lambda out, *rest: outputs.append(os.path.basename(out)) or out)
    if lacking == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    elif lacking == "a torch with CUDA":
        exists = os.path.exists
        monkeypatch.setattr(os.path, "exists", lambda p: not str(p).endswith("libc10_cuda.so") and exists(p))
    elif lacking:
        monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build.build() == build.LIB
    assert outputs[0] == "libsvdq_b200.so" and len(outputs) == (1 if lacking else 2)
    err = capsys.readouterr().err
    assert (f"not built: no {lacking}" in err) if lacking else err == ""


def test_a_module_of_another_torch_or_python_is_not_used(monkeypatch):
    """After an upgrade of either the old file is neither loaded nor taken as built."""
    import sysconfig

    import torch

    from bit_w4a4_quantized_token_b200 import build, layer

    here, config = build.front_path(), sysconfig.get_config_var
    outputs = []
    monkeypatch.setattr(build, "_compile", lambda out, *rest: outputs.append(out) or out)
    monkeypatch.setattr(layer, "_front", layer._Unloaded())
    for change in ("torch", "python"):
        with monkeypatch.context() as m:
            if change == "torch":
                m.setattr(torch, "__version__", "99.0.0")
            else:
                m.setattr(sysconfig, "get_config_var", lambda name: ".cpython-399-x86_64-linux-gnu.so"
                          if name == "EXT_SUFFIX" else config(name))
            build.build()
            assert outputs[-1] != here and not os.path.exists(outputs[-1])
            with pytest.raises(ImportError, match="not built"):
                layer.quantize_act_w8a8(torch.zeros(4, 32), layer.PackedWeightW8A8(8, 32, None, None, None, None))
    build.build()
    assert outputs[-1] == here
    with pytest.raises(ValueError, match="x:"):
        layer.quantize_act_w8a8(torch.zeros(4, 32), layer.PackedWeightW8A8(8, 32, None, None, None, None))


def test_no_row_kernel_that_no_call_reaches():
    """The fp32 norm holds at most one vector of eight a thread in registers: wider rows are 16 KB, the ring's."""
    import re

    from bit_w4a4_quantized_token_b200 import build

    names = subprocess.check_output(["nm", build.LIB], text=True)
    held = {tuple(map(int, m)) for m in re.findall(r"quantize_rows_w8_kernelILi(\d)ELb(\d)ELi(\d)E", names)}
    bf16, f16, f32 = range(3)
    assert held == {(t, norm, v) for t in (bf16, f16, f32) for norm in (0, 1) for v in (1, 2)} - {(f32, 1, 2)}
