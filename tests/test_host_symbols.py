"""Host functions of the kernels' files (CPU): templates are weak symbols, and of two
with one name and signature in two files the linker keeps one, silently, whatever the
other did."""
import os
import shutil
import subprocess

import pytest

from activation_sparse_moe_gb300 import build as hsbuild


@pytest.mark.skipif(shutil.which("nm") is None, reason="no nm")
def test_no_template_of_the_library_is_defined_in_two_files():
    hsbuild.build()
    where = {}
    for src in hsbuild.sources():
        obj = os.path.join(hsbuild.BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        if not os.path.exists(obj):
            hsbuild.build(force=True)
        out = subprocess.run(["nm", "--defined-only", obj], capture_output=True, text=True, check=True).stdout
        for line in out.splitlines():
            kind, name = line.split()[-2:]
            if kind in "Ww" and name.startswith("_ZN2hs"):
                where.setdefault(name, []).append(os.path.basename(src))
    assert any("launch_decode8" in k for k in where) and any("launch_prefillI" in k for k in where)
    twice = {k: v for k, v in where.items() if len(v) > 1}
    assert not twice, twice
