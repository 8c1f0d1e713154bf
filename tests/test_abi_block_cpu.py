"""Host side of the entry points around the experts' products (no GPU): from plain C, under sanitizers, and what the Python
module refuses before a call."""

import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from grouped_expert_ffn_router_amd import binding as B, block, build, runner

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "grouped_expert_ffn_router_amd")
NATIVE = os.path.join(ROOT, "tests", "native")


def _run(cmd, **kw):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, **kw)
    assert r.returncode == 0, " ".join(cmd) + "\n" + r.stdout[-3000:]
    return r.stdout


def test_the_entry_points_from_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    B.lib()  # raises if the library was not built
    exe = str(tmp_path / "block_c")
    _run([gcc, "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
          os.path.join(NATIVE, "abi_c_block_check.c"), "-L", PKG, "-lmoe", f"-Wl,-rpath,{PKG}", "-o", exe])
    assert _run([exe], timeout=60).startswith("ok")


def test_the_host_code_under_address_and_undefined_behaviour_sanitizers(tmp_path):
    """The unit that holds the whole C ABI (block/entry.hip) and the operators' host code (launch rules, workspace sizes),
    sanitized on the host side only, under every C client."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    clang = "/opt/rocm/llvm/bin/clang"
    if not (os.path.exists(hipcc) and os.path.exists(clang)):
        pytest.skip("hipcc / clang not available")
    kernels_o = os.path.join(PKG, "_build", "kernels.o")
    if not os.path.exists(kernels_o):
        pytest.skip("build the library first")
    csrc = os.path.join(PKG, "csrc")
    san = ["-Xarch_host", "-fsanitize=address,undefined", "-Xarch_host", "-fno-omit-frame-pointer"]

    def compile_one(name):
        obj = str(tmp_path / (os.path.basename(name) + ".o"))
        _run([hipcc, "--offload-arch=gfx950", "-O1", "-g", "-fPIC", "-std=c++17", "-Wno-unused-function", "-Xclang",
              "-target-feature", "-Xclang", "-packed-fp32-ops", *san, "-I", os.path.join(ROOT, "include"), "-I", csrc, "-c",
              os.path.join(csrc, name), "-o", obj])
        return obj

    names = [n for n in build.SOURCES if n != "kernels.hip"]
    with ThreadPoolExecutor(len(names)) as ex:
        objects = list(ex.map(compile_one, names))
    _run([hipcc, "--offload-arch=gfx950", "-shared", *san, "-o", str(tmp_path / "libmoe.so"), *objects, kernels_o])
    env = dict(os.environ, ASAN_OPTIONS="abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    for name in ("abi_c_block_check", "abi_c_ops_check", "abi_c_check"):
        exe = str(tmp_path / name)
        _run([clang, "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-g", "-fsanitize=address,undefined",
              "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include"), os.path.join(NATIVE, name + ".c"), "-L",
              str(tmp_path), "-lmoe", f"-Wl,-rpath,{tmp_path}", "-o", exe])
        out = _run([exe], env=env, timeout=120)
        assert out.startswith("ok"), out[-2000:]
        assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out


def _rows8(rows, cols):
    cb, sb = B.mx8_strides(cols)
    return block.Mx8Rows(torch.zeros((rows, cb), dtype=torch.uint8), torch.zeros((rows, sb), dtype=torch.uint8), cols)


def test_tensors_off_the_gpu_are_refused():
    x, w = torch.zeros((4, 64)), torch.ones(64)
    rule = block.RouterRule(2)
    for call in (lambda: block.rms_norm(x, w), lambda: block.rms_norm_backward(x, x, w), lambda: block.mx8_quantize(x),
                 lambda: block.mx8_dequantize(_rows8(4, 64)), lambda: block.select_experts(x, rule),
                 lambda: block.select_experts_backward(x[:, :2], x[:, :2], x[:, :2].int(), x, rule),
                 lambda: block.swiglu_checkpoint(x), lambda: block.swiglu_backward(x, _rows8(4, 128))):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_types_shapes_and_rules_are_refused():
    x, w = torch.zeros((4, 64)), torch.ones(64)
    with pytest.raises(TypeError):
        block.rms_norm(x.half(), w)
    with pytest.raises(TypeError):
        block.rms_norm(x, w.half())
    with pytest.raises(ValueError):
        block.rms_norm(x, w, form="fp8")
    with pytest.raises(TypeError):
        block.mx8_quantize(x.double())
    with pytest.raises(TypeError):
        block.mx8_dequantize(_rows8(4, 64), torch.float16)
    with pytest.raises(TypeError):
        block.mx8_dequantize(runner.MxRows(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 16), dtype=torch.uint8), 64))
    with pytest.raises(ValueError):
        block.swiglu_checkpoint(torch.zeros((4, 96)))
    with pytest.raises(ValueError):
        block.swiglu_checkpoint(torch.zeros((1, 1, 4, 64)))
    with pytest.raises(ValueError):
        block.swiglu_backward(torch.zeros((4, 32)), _rows8(4, 32))
    with pytest.raises(TypeError):
        block.swiglu_backward(torch.zeros((4, 32)), x)
    with pytest.raises(ValueError):
        block.select_experts(x.bfloat16(), block.RouterRule(2))
    with pytest.raises(ValueError):
        block.RouterRule(2, score="relu")
    with pytest.raises(ValueError):
        _rows8(4, 64)[0:2].__class__(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 16), dtype=torch.uint8), 64)
    with pytest.raises(B.MoeError):   # not a multiple of 32
        _rows8(4, 40)
    with pytest.raises(AttributeError):   # a rule does not change
        block.RouterRule(2).top_k = 3


def test_rows_of_eight_bits_are_not_taken_for_rows_of_four():
    assert not isinstance(_rows8(4, 64), runner.MxRows)
    with pytest.raises(TypeError):
        runner.mx_gemm(_rows8(4, 64), _rows8(4, 64))
    with pytest.raises(TypeError):
        runner.mx_dequantize(_rows8(4, 64))
    half = _rows8(4, 64)[1:3]
    assert isinstance(half, block.Mx8Rows) and half.shape == (2, 64)
