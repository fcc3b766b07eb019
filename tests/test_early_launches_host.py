"""CPU test of the sources: kernels that may begin while the one before them runs read nothing through the read-only cache, since
that one may have written it (csrc/kvarn_block_dev.cuh, read)."""
import os
import re

from quantized_kv_cache_seal_gb300 import build


def test_early_kernels_read_by_plain_loads():
    seen = 0
    for name in build.SOURCES:
        text = re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, name)).read())
        if "launch_behind(" in text:
            seen += 1
            assert "__ldg(" not in text and "__restrict__" not in text and "ld.global.nc" not in text, name
            assert "sealed_tile(" not in text, name  # looks the pool slot up that way
    assert seen >= 5
