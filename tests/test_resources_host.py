"""CPU check of the built library: the attention kernels keep all their values
in registers.  (One that spilled some of them gave wrong sums, and was dropped.)"""
import glob
import os
import re
import shutil
import subprocess

import pytest

import kv_cache_compression_decode_amd as kvc

LLVM = "/opt/rocm/llvm/bin"
pytestmark = pytest.mark.skipif(not os.path.exists(LLVM + "/llvm-readelf"),
                                reason="no tools to read the library's notes with")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Each kernel's name and the compiler's report of it."""
    if not os.path.exists(kvc.LIB_PATH):
        from kv_cache_compression_decode_amd import build

        build.build()
    at = tmp_path_factory.mktemp("notes")
    shutil.copy(kvc.LIB_PATH, at / "lib.so")
    subprocess.run([LLVM + "/llvm-objdump", "--offloading", "lib.so"], cwd=at, check=True,
                   stdout=subprocess.DEVNULL)
    found = {}
    for f in glob.glob(str(at / "*gfx950")):
        notes = subprocess.run([LLVM + "/llvm-readelf", "--notes", f], check=True,
                               capture_output=True, text=True).stdout
        # a kernel's entry begins with a dash at the list's depth
        for entry in re.split(r"\n  - ", notes)[1:]:
            name = re.search(r"\.name: +(\S+)", entry)
            if name:
                found[name.group(1)] = {k: int(v) for k, v in re.findall(
                    r"\.(\w+_spill_count|private_segment_fixed_size|\w*vgpr_count): +(\d+)",
                    entry)}
    return found


@pytest.mark.parametrize("kind", ["k_attend_rows", "k_attend_few", "k_attend_tile",
                                  "k_attend_tree", "join"])
def test_nothing_is_spilled(kernels, kind):
    mine = {n: k for n, k in kernels.items() if "k_attend" in n and kind in n}
    assert len(mine) >= 12  # three pairs of types, four head dimensions
    assert any("Li256E" in n for n in mine)
    for name, k in mine.items():
        assert k["vgpr_spill_count"] == 0 and k["private_segment_fixed_size"] == 0, name
        assert k["vgpr_count"] <= 512, name
