"""The host code of linear attention and layer norm built with the address and undefined-behaviour sanitizers and run
on the CPU with stub launchers (tests/sanitize/attn_driver.cpp)."""
import os

import pytest

from test_sanitizers import CSRC, ENV, HERE, ROCM, ROOT, _run


@pytest.mark.skipif(not os.path.exists(os.path.join(ROCM, "bin", "hipcc")), reason="needs the ROCm toolchain")
def test_attn_host_code_under_sanitizers(tmp_path):
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    objs = []
    for src in (os.path.join(CSRC, "abi_attn.cpp"), os.path.join(HERE, "attn_stubs.cpp"),
                os.path.join(HERE, "attn_driver.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([os.path.join(ROCM, "bin", "hipcc"), "-O1", "-g", "-std=c++17", "-fPIC"] + san + inc + ["-c", src, "-o", obj])
        objs.append(obj)
    exe = str(tmp_path / "attn_driver")
    _run([os.path.join(ROCM, "llvm", "bin", "clang++"), "-fsanitize=address,undefined"] + objs +
         ["-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-Wl,-rpath," + os.path.join(ROCM, "lib"), "-o", exe])
    r = _run([exe], env=ENV)
    assert "all host paths behaved" in r.stdout, r.stdout
    assert "runtime error" not in r.stderr
