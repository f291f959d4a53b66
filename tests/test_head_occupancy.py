"""The built product kernels hold as many blocks a CU as their plan counts on:
a SIMD has 512 registers a lane for the waves of all of them, a CU 160 KB of
LDS.  Read from the built library's own kernel descriptions."""
import os
import re
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "histogram_gradient_boosted_amd")
READELF = "/opt/rocm/llvm/bin/llvm-readelf"

pytestmark = pytest.mark.skipif(not os.path.exists(READELF), reason="llvm-readelf not found")


def kernels(folder):
    """Name and registers of each device kernel of libhgb.so (of a lane, both kinds of them)."""
    lib = os.path.join(PKG, "libhgb.so")
    if not os.path.exists(lib):
        pytest.fail("libhgb.so not built: run __graft_entry__.build()")
    data = open(lib, "rb").read()
    found = {}
    for bundle in re.finditer(b"__CLANG_OFFLOAD_BUNDLE__", data):   # of each source file: the count, then offset, size and target
        at, count = bundle.start(), struct.unpack_from("<Q", data, bundle.start() + 24)[0]
        entry = at + 32
        for _ in range(count):
            offset, size, name = struct.unpack_from("<QQQ", data, entry)
            target = data[entry + 24:entry + 24 + name]
            entry += 24 + name
            if b"gfx950" not in target:
                continue
            code = folder / f"{at}.co"
            code.write_bytes(data[at + offset:at + offset + size])
            notes = subprocess.run([READELF, "--notes", str(code)], capture_output=True, text=True, check=True).stdout
            found.update((n, int(v)) for n, v in re.findall(r"\.name: +(\S+)\n(?:(?!\.name:).*\n)*? +\.vgpr_count: +(\d+)", notes))
    return found


def tiles():
    """(rows, columns) -> blocks a CU, as planned."""
    text = open(os.path.join(PKG, "csrc", "hgb_vector_head_plan.h")).read()
    line = re.search(r"constexpr Tile kTiles\[\] = \{(.*)\};", text).group(1)
    return {(int(m), int(n)): int(blocks) for m, n, blocks in re.findall(r"\{(\d+), (\d+), \d+, (\d+),", line)}


def test_registers_hold_the_planned_blocks(tmp_path):
    plan, seen = tiles(), set()
    for name, registers in kernels(tmp_path).items():
        tile = re.search(r"k_product\w+?Li(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E", name)
        if not tile:
            continue
        rows, columns, wm, wn = (int(v) for v in tile.groups())
        waves = plan[rows, columns] * wm * wn / 4   # of a SIMD
        assert (registers + 7) // 8 * 8 * waves <= 512, (name, registers)
        seen.add((rows, columns))
    assert seen == set(plan) and len(plan) == 4
