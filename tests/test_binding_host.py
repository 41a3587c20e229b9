"""CPU tests of the compiled binding's own parts (csrc/binding.cpp)."""
import os
import subprocess

from fp8_block_scaled_gemm_amd import build

DEVICE_PROGRAM = r"""
// on_device.h against a runtime whose calls fail on demand
#include "on_device.h"
#include <cstdio>
#include <cstdlib>
static int current = 1, get_fails = 0, set_fails = 0, sets = 0;
extern "C" hipError_t hipGetDevice(int* d) { *d = current; return get_fails ? hipErrorNoDevice : hipSuccess; }
extern "C" hipError_t hipSetDevice(int d) {
    ++sets;
    if (set_fails) return hipErrorInvalidDevice;
    current = d;
    return hipSuccess;
}
static bool refused(int index) {
    try {
        const OnDevice on(index);
        if (current != index) std::exit(9);  // went on, on another GPU
        return false;
    } catch (const std::exception&) { return true; }
}
int main() {
    if (refused(1) || sets != 0) return 1;               // current already
    if (refused(3) || sets != 2 || current != 1) return 2;  // made current, and back
    set_fails = 1;
    if (!refused(3) || current != 1 || sets != 3) return 3;
    if (refused(1)) return 4;
    set_fails = 0, get_fails = 1;
    if (!refused(1)) return 5;
    std::puts("ok");
    return 0;
}
"""


def test_a_gpu_that_cannot_be_made_current_is_an_error(tmp_path):
    src, exe = tmp_path / "on_device.cpp", tmp_path / "on_device"
    src.write_text(DEVICE_PROGRAM)
    rocm = os.path.dirname(os.path.dirname(build.hipcc()))
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-D__HIP_PLATFORM_AMD__", f"-I{build.CSRC}",
                    f"-I{rocm}/include", str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True)
    assert got.returncode == 0 and got.stdout == "ok\n", got


def test_workspaces_have_a_size_that_a_caller_can_ask_for():
    import ctypes

    import fp8_block_scaled_gemm_amd as dg

    lib, n = dg.load_library(), ctypes.c_int64()
    for name, sizes, bad in (("dg_moe_mlp_fp8_workspace", (4, 2, 8, 256, 128), (4, 2, 8, 200, 128)),
                             ("dg_fp8_gemm_nt_lora_workspace", (64, 264, 512, 4, 16), (64, 264, 512, 4, 12))):
        assert name in dg.__all__
        assert getattr(lib, name)(*sizes, ctypes.byref(n)) == 0
        assert getattr(dg, name)(*sizes) == n.value > 0
        try:
            getattr(dg, name)(*bad)
        except dg.DGError as e:
            assert name in str(e)
        else:
            raise AssertionError(name)
    assert dg.dg_fp8_gemm_nt_lora_workspace(0, 264, 512, 4, 16) == 0


def test_a_binding_that_does_not_compile_leaves_the_library_in_its_place(tmp_path, monkeypatch):
    lib, binding = tmp_path / "libdgfp8.so", tmp_path / "_binding.so"
    for f in (lib, binding):
        f.write_bytes(b"before")
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "BINDING", str(binding))
    monkeypatch.setattr(build, "SOURCES", ["quantize.hip"])
    monkeypatch.setenv("CXX", "false")
    try:
        build.build()
    except subprocess.CalledProcessError:
        pass
    else:
        raise AssertionError("a host compiler that fails went unnoticed")
    assert lib.read_bytes() == b"before" and binding.read_bytes() == b"before"
    assert build.build_library() == str(lib)  # which needs no host compiler
    assert lib.read_bytes()[:4] == b"\x7fELF" and binding.read_bytes() == b"before"
