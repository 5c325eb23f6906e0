"""What the built library's own GPU code must hold, read from its disassembly (no GPU).

A copy into LDS takes its place there from M0, and the instruction that writes M0 needs one wait state
before such a copy: at least one other instruction has to stand between the two. The compiler sees to that
for its own copies, not inside inline assembly."""
import os
import re
import struct
import subprocess

import pytest

import chunked_weight_sequence_amd as ttt

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _code_objects():
    """The gfx950 code objects of the library, one per source."""
    data = open(ttt.library_path, "rb").read()
    for m in re.finditer(MAGIC, data):
        at = m.start() + len(MAGIC)
        (n,) = struct.unpack_from("<Q", data, at)
        at += 8
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", data, at)
            name = data[at + 24:at + 24 + length]
            at += 24 + length
            if b"gfx950" in name and size:
                yield data[m.start() + offset:m.start() + offset + size]


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no disassembler")
def test_copies_into_lds_wait_for_m0(tmp_path):
    copies = 0
    for i, code in enumerate(_code_objects()):
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(path)], capture_output=True, text=True,
                              check=True).stdout
        before = ""
        for line in text.split("\n"):
            op = line.split("//")[0].strip()
            if not op:
                continue
            if re.match(r"(global|buffer|scratch)_load_lds|buffer_load.*\blds\b", op):
                copies += 1
                assert not re.match(r"s_\w+\s+m0\b", before), (before, op)
            before = op
    assert copies > 100
