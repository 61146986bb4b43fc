"""The form of the wide buffer stores in the built library's gfx950 code (CPU only).

A store of 12 or 16 bytes reads its data registers over more than one cycle, and an instruction right
behind it may overwrite them.  The compiler keeps the two apart where the store's scalar offset is a
constant, and not where it is a register; there stores of the new values were seen on gfx950.  So no
kernel may store 12 or 16 bytes through a buffer resource with a register as the scalar offset."""

import os
import re
import struct
import subprocess

import pytest

import mxfp4_microscaled_quantization_amd as mxq

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
WIDE = re.compile(r"buffer_store_(?:format_xyzw?|dwordx[34])\s+(.*)")


def _code_objects(blob):
    """The gfx950 code objects in the offload bundles of a shared library: after the magic, the number of
    entries, then (offset, size, length of the name, name) of each."""
    at = blob.find(MAGIC)
    while at >= 0:
        count, = struct.unpack_from("<Q", blob, at + len(MAGIC))
        entry = at + len(MAGIC) + 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", blob, entry)
            name = blob[entry + 24:entry + 24 + length]
            entry += 24 + length
            if b"gfx950" in name and size:
                yield blob[at + offset:at + offset + size]
        at = blob.find(MAGIC, at + 1)


def scalar_offset(operands):
    """The scalar offset of a buffer store's operands: data, [address,] resource, offset and modifiers."""
    fields = [f.strip() for f in operands.split("//")[0].split(",")]
    assert re.match(r"s\[\d+:\d+\]|off", fields[2]) or re.match(r"s\[\d+:\d+\]", fields[1]), operands
    return fields[-1].split()[0]


def test_operand_parser():
    assert scalar_offset("v[0:3], v11, s[0:3], 0 offen nt") == "0"
    assert scalar_offset("v[0:3], v11, s[0:3], s7 offen offset:16") == "s7"
    assert scalar_offset("v[0:3], off, s[0:3], 0 // 0000: E0") == "0"
    assert WIDE.search("  buffer_store_dwordx4 v[0:3], v1, s[0:3], m0 offen") and not WIDE.search("buffer_store_dwordx2 v[0:1], v1")


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="llvm-objdump not found")
def test_no_wide_buffer_store_has_a_register_as_its_scalar_offset(tmp_path):
    with open(mxq.LIB_PATH, "rb") as f:
        objects = list(_code_objects(f.read()))
    assert objects
    seen = 0
    for i, code in enumerate(objects):
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(path)], capture_output=True, text=True, check=True).stdout
        assert "s_endpgm" in text
        for m in WIDE.finditer(text):
            seen += 1
            assert scalar_offset(m.group(1)) == "0", m.group(0)
    assert seen > 0   # the head norm and the rotation before MXFP4 store 16 bytes this way
