"""Rules that the sources of the cache operators keep, read from the files."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "causal_gqa_attention_rmsnorm_gb300",
                    "csrc")


def code(path):
    """The file without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


def test_no_non_coherent_load_of_what_the_kernel_before_may_write():
    """The grids are resident while the kernel before them still runs; ld.global.nc
    is for memory that is read-only as long as the grid lives."""
    files = sorted(glob.glob(os.path.join(CSRC, "cache*.cu*")))
    assert len(files) >= 6
    for f in files:
        found = re.findall(r"__ldg\b|ld\.global(?:\.\w+)*\.nc|__restrict__", code(f))
        assert not found, (os.path.basename(f), found)
