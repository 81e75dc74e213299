"""What the library's own gfx950 code has to observe and the compiler cannot see to, because it stands in inline
assembly.  The code objects of libforge.so are listed with the toolchain's disassembler; no GPU needed."""
import os
import re
import struct
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", "/opt/rocm/lib/llvm/bin/llvm-objdump") if os.path.exists(p)), None)
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
WRITES_M0 = re.compile(r"^s_\w+ m0\b")
COPY = re.compile(r"^buffer_load_\w+ .*\blds$")


def code_objects(path):
    """The gfx950 code objects of a library's offload bundles."""
    data = open(path, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        p, n = at + 32, struct.unpack_from("<Q", data, at + 24)[0]
        for _ in range(n if n < 16 else 0):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            if b"gfx950" in data[p + 24:p + 24 + length] and size:
                yield data[at + offset:at + offset + size]
            p += 24 + length
        at = data.find(MAGIC, at + 24)


def copies_too_early(lines):
    """(copies to LDS, those that directly follow the instruction that writes M0): gfx9 wants one wait state between
    them.  `lines`: a disassembly."""
    copies = early = 0
    last = ""
    for line in lines:
        if not line.startswith("\t"):
            continue
        text = line.split("//")[0].strip()
        if COPY.match(text):
            copies += 1
            early += bool(WRITES_M0.match(last))
        last = text
    return copies, early


def test_the_rule_itself():
    good = ["\ts_mov_b32 m0, s4     // 00: BEFC0004", "\ts_nop 0    // 04: BF800000", "\tbuffer_load_dwordx4 v1, s[0:3], 0 offen lds   // 08:"]
    assert copies_too_early(good) == (1, 0)
    assert copies_too_early([good[0], good[2]]) == (1, 1)
    assert copies_too_early(["\ts_add_u32 m0, s4, 0x400 // 00:", "\tbuffer_load_dword v1, s[0:3], 0 offen lds // 08:"]) == (1, 1)
    assert copies_too_early([good[0], "\tbuffer_load_dword v1, v2, s[0:3], 0 offen // 08:"]) == (0, 0)


@pytest.mark.skipif(OBJDUMP is None, reason="no disassembler in this toolchain")
def test_copies_to_lds_wait_for_m0(tmp_path):
    import optimizer_step_weight_amd as forge
    if not os.path.exists(forge.LIB_PATH):
        from optimizer_step_weight_amd import _build
        _build.build(verbose=False)

    def check(i_and_code):
        i, code = i_and_code
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        with subprocess.Popen([OBJDUMP, "-d", "--no-show-raw-insn", str(path)], stdout=subprocess.PIPE, text=True) as p:
            found = copies_too_early(p.stdout)
        assert p.returncode == 0
        return found

    with ThreadPoolExecutor(4) as ex:
        found = list(ex.map(check, enumerate(code_objects(forge.LIB_PATH))))
    assert sum(n for n, _ in found) > 1000     # the contractions' copies
    assert sum(n for _, n in found) == 0
