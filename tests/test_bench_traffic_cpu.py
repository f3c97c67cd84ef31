"""The recorded DRAM traffic of a decode launch counts only while the kernel's
source is the one it was captured from."""
import os
import re
import shutil

import bench


def test_hash_covers_the_kernel_and_changes_with_it(tmp_path, monkeypatch):
    csrc = os.path.join("int2_kv_cache_rotate_b200", "csrc")
    defined = [n for n in os.listdir(os.path.join(bench.ROOT, csrc))
               if re.search(r"__global__[^;{]*decode_heads_kernel\(", open(os.path.join(bench.ROOT, csrc, n)).read())]
    assert defined and set(defined) <= set(bench.KERNEL_SOURCES)
    shutil.copytree(os.path.join(bench.ROOT, csrc), tmp_path / csrc)
    before = bench.kernel_source_hash()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_source_hash() == before
    for name in bench.KERNEL_SOURCES:
        with open(tmp_path / csrc / name, "a") as f:
            f.write("// changed\n")
        assert bench.kernel_source_hash() != before
        before = bench.kernel_source_hash()
