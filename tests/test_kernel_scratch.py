"""No kernel of the grouped products or of 4-bit weights keeps anything in scratch memory: an
array that the compiler puts there costs a load and a wait for every load in flight, which a
loop that runs loads ahead cannot afford. Read from the metadata of the built library; no
kernel runs."""
import os
import re
import shutil
import struct
import subprocess

import pytest

from token_choice_routing_amd import LIB_PATH

READELF = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-readelf")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _code_objects(data):
    """Device code of a library: every bundle lists (offset, size, target) of its parts."""
    at = data.find(MAGIC)
    while at >= 0:
        count, = struct.unpack_from("<Q", data, at + len(MAGIC))
        p = at + len(MAGIC) + 8
        for _ in range(count):
            offset, size, n = struct.unpack_from("<QQQ", data, p)
            target = data[p + 24:p + 24 + n]
            p += 24 + n
            if b"gfx950" in target and size:
                yield data[at + offset:at + offset + size]
        at = data.find(MAGIC, p)


def _scratch(tmp_path):
    """Bytes of scratch memory a lane, by kernel."""
    out = {}
    with open(LIB_PATH, "rb") as f:
        data = f.read()
    for i, elf in enumerate(_code_objects(data)):
        path = tmp_path / f"{i}.elf"
        path.write_bytes(elf)
        notes = subprocess.run([READELF, "--notes", str(path)], capture_output=True, text=True, check=True).stdout
        names = re.findall(r"^\s*\.name:\s+'?(_Z\w+)'?$", notes, re.M)
        sizes = re.findall(r"^\s*\.private_segment_fixed_size:\s+(\d+)$", notes, re.M)
        assert len(names) == len(sizes)
        out.update(zip(names, map(int, sizes)))
    return out


@pytest.mark.skipif(not shutil.which(READELF), reason="no llvm-readelf")
def test_grouped_kernels_keep_nothing_in_scratch(tmp_path):
    kernels = _scratch(tmp_path)
    mine = {n: b for n, b in kernels.items() if "grouped_mm_" in n or "weights4_" in n}
    assert len(mine) >= 40 and any("grouped_mm_tiles" in n for n in mine) and any("weights4_" in n for n in mine)
    assert {n: b for n, b in mine.items() if b} == {}
