"""Host side of the MX-FP4 and few-token entry points (no GPU): from plain C, under sanitizers, and with arbitrary dims."""

import ctypes
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
from hypothesis import given, settings, strategies as st

from grouped_expert_ffn_router_amd import binding as B
from workload import configs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "grouped_expert_ffn_router_amd")
CHECK = os.path.join(ROOT, "tests", "native", "abi_c_ops_check.c")


def _run(cmd, **kw):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, **kw)
    assert r.returncode == 0, " ".join(cmd) + "\n" + r.stdout[-3000:]
    return r.stdout


def test_the_entry_points_from_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    B.lib()  # raises if the library was not built
    exe = str(tmp_path / "ops_c")
    _run([gcc, "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), CHECK, "-L", PKG,
          "-lmoe", f"-Wl,-rpath,{PKG}", "-o", exe])
    assert _run([exe], timeout=60).startswith("ok")


def test_the_whole_c_abi_under_address_and_undefined_behaviour_sanitizers(tmp_path):
    """The unit that holds the whole C ABI (ops/entry.hip, which includes api.hip) and the host code of the operators'
    kernels (ops/mx.hip, ops/few.hip: workspace layout, launch rules), sanitized on the host side only, under both C
    clients."""
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
        obj = str(tmp_path / (name + ".o"))
        _run([hipcc, "--offload-arch=gfx950", "-O1", "-g", "-fPIC", "-std=c++17", "-Wno-unused-function", "-Xclang",
              "-target-feature", "-Xclang", "-packed-fp32-ops", *san, "-I", os.path.join(ROOT, "include"), "-I", csrc, "-c",
              os.path.join(csrc, "ops", name + ".hip"), "-o", obj])
        return obj

    with ThreadPoolExecutor(3) as ex:
        objects = list(ex.map(compile_one, ("entry", "mx", "few")))
    _run([hipcc, "--offload-arch=gfx950", "-shared", *san, "-o", str(tmp_path / "libmoe.so"), *objects, kernels_o])
    env = dict(os.environ, ASAN_OPTIONS="abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    for name in ("abi_c_ops_check", "abi_c_check"):
        exe = str(tmp_path / name)
        _run([clang, "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-g", "-fsanitize=address,undefined",
              "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include"),
              os.path.join(ROOT, "tests", "native", name + ".c"), "-L", str(tmp_path), "-lmoe", f"-Wl,-rpath,{tmp_path}",
              "-o", exe])
        out = _run([exe], env=env, timeout=120)
        assert out.startswith("ok"), out[-2000:]
        assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out


_FIELDS = [f for f, _ in B.Dims._fields_]
_INT32 = st.one_of(st.integers(-3, 70000), st.sampled_from([-2**31, -1, 0, 1, 2**31 - 1, 2**30, 65536, 1 << 24]))


@settings(max_examples=400, deadline=None, derandomize=True)
@given(base=st.sampled_from([3, 5, "mini_bf16", "mini_f32"]), tokens=st.integers(0, 64), one_rank=st.booleans(),
       edits=st.lists(st.tuples(st.sampled_from(_FIELDS), _INT32), max_size=3))
def test_workspace_sizes_of_any_dims(base, tokens, one_rank, edits):
    """moe_mx_workspace_size and moe_few_workspace_size on dims with up to three fields at arbitrary int32 values: a
    documented code, and sizes that hold what the formulas need in exact integers."""
    d = B.make_dims(configs.get(base))
    few = B.Dims.from_buffer_copy(d)
    few.tokens = tokens
    if one_rank:
        few.n_ranks, few.my_rank = 1, 0
    for f, v in edits:
        setattr(d, f, v)
        setattr(few, f, v)
    n = ctypes.c_size_t()
    codes = {B.MOE_OK, B.MOE_EINVAL, B.MOE_EDTYPE}
    rc = B.lib().moe_few_workspace_size(ctypes.byref(few), ctypes.byref(n))
    assert rc in codes and (rc == B.MOE_OK or B.last_error())
    if rc == B.MOE_OK:
        T, X = few.tokens, few.n_experts // few.n_ranks
        need = T * (4 * few.n_experts + 4 * X + 8 * few.latent + 4 * few.top_k * few.expert_hidden
                    + 4 * few.shared_experts * few.shared_hidden)
        shares = 64 * 4 * 512 * few.latent   # of the down product, at most
        padding = 16 * 256 + 32 * X + 4 * few.latent
        assert need <= n.value <= need + shares + padding
        assert (n.value == 0) == (T == 0)
    rc = B.lib().moe_mx_workspace_size(ctypes.byref(d), ctypes.byref(n))
    assert rc in codes and (rc == B.MOE_OK or B.last_error())
    if rc == B.MOE_OK:
        _, rcap, _ = B.capacity(d)
        rows = d.wave_rows if d.wave_rows > 0 else d.n_experts // d.n_ranks // d.waves * rcap
        live = d.live_waves if d.live_waves > 0 else d.waves
        scales = lambda cols: -(-cols // 512) * 16  # noqa: E731
        parts = [rows * d.latent // 2, rows * scales(d.latent), rows * d.expert_hidden // 2, rows * scales(d.expert_hidden)]
        assert n.value == live * sum(-(-p // 256) * 256 for p in parts)
