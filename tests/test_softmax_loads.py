"""The loads from memory into LDS that softmax attention's kernels write out as assembly: the compiler looks into none of it, so
that the wait states that gfx950 asks for have to be written out too. Read in the code that the build made of the sources."""
import os
import re
import struct
import subprocess

import pytest

from selective_state_space_82_amd import build

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
OBJCOPY = "/opt/rocm/llvm/bin/llvm-objcopy"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(lib, folder):
    """The gfx950 code objects of a library, one for each source."""
    section = os.path.join(folder, "fatbin")
    subprocess.run([OBJCOPY, f"--dump-section=.hip_fatbin={section}", lib, os.path.join(folder, "copy")], check=True)
    data = open(section, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        (n,) = struct.unpack_from("<Q", data, at + len(MAGIC))
        p = at + len(MAGIC) + 8
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            name = data[p + 24:p + 24 + length]
            p += 24 + length
            if b"gfx950" in name:
                yield data[at + offset:at + offset + size]
        at = data.find(MAGIC, at + 1)


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Instructions of each kernel with a load into LDS."""
    if not (os.path.exists(OBJDUMP) and os.path.exists(OBJCOPY)):
        pytest.skip("needs the ROCm toolchain")
    folder = str(tmp_path_factory.mktemp("code"))
    found = {}
    for i, code in enumerate(code_objects(build.LIB, folder)):
        if b"softmax_" not in code:
            continue
        path = os.path.join(folder, f"{i}.co")
        with open(path, "wb") as f:
            f.write(code)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", path], check=True, capture_output=True, text=True).stdout
        for part in re.split(r"^[0-9a-f]+ <", text, flags=re.M)[1:]:
            name, body = part.split(">:", 1)
            lines = [s.split("//")[0].strip() for s in body.splitlines()]
            lines = [s for s in lines if s and not s.endswith(":")]
            if any(re.match(r"buffer_load.*\blds$", s) for s in lines):
                found[name] = lines
    return found


def states(s):
    """Wait states that an instruction is good for."""
    m = re.match(r"s_nop (\w+)", s)
    return int(m[1], 0) + 1 if m else 1


def scalars(operand):
    """Scalar registers of an operand: s7 or s[4:7]."""
    m = re.fullmatch(r"s(\d+)|s\[(\d+):(\d+)\]", operand)
    if not m:
        return set()
    return {int(m[1])} if m[1] else set(range(int(m[2]), int(m[3]) + 1))


def test_there_are_such_loads(kernels):
    assert any("softmax_fwd" in n for n in kernels) and any("softmax_dq" in n for n in kernels) and \
        any("softmax_dkv" in n for n in kernels)


def test_wait_states_before_loads_into_lds(kernels):
    """One between a scalar write of m0 and the load that takes its place in LDS from it; five between a vector instruction's write of a
    scalar register (readfirstlane, a spilled register's readlane) and the load that reads it."""
    for name, lines in kernels.items():
        for i, s in enumerate(lines):
            if not re.match(r"buffer_load.*\blds$", s):
                continue
            reads = set().union(*(scalars(x) for x in re.findall(r"s\d+|s\[\d+:\d+\]", s)))
            waited, m0 = 0, None
            for t in reversed(lines[max(0, i - 8):i]):
                if m0 is None and re.match(r"s_\w+ m0,", t):
                    m0 = waited
                if waited < 5 and t.startswith("v_"):
                    written = scalars(t.split(None, 1)[1].split(",")[0].strip()) if " " in t else set()
                    assert not written & reads, (name, t, s)
                waited += states(t)
            assert m0 is not None and m0 >= 1, (name, lines[max(0, i - 8):i + 1])


def test_nothing_else_uses_m0(kernels):
    """The compiler keeps nothing in m0 across such a load."""
    for name, lines in kernels.items():
        for i, s in enumerate(lines):
            if re.search(r"\bm0\b", s):
                assert re.match(r"s_mov_b32 m0, s\d+$|s_mov_b32 m0, (0x)?[0-9a-f]+$", s), (name, s)
                assert any(re.match(r"buffer_load.*\blds$", t) for t in lines[i + 1:i + 3]), (name, lines[i:i + 3])
