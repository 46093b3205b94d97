"""Rules that the sources of the 8-bit projections keep, read from the files."""
import os
import re

from test_cache_sources import CSRC, code


def source(name):
    return code(os.path.join(CSRC, name))


def test_what_a_cta_writes_is_released_to_the_other_cta_at_cluster_scope():
    """The scales of a pair's odd CTA are written by its threads and read by copies that the
    even CTA issues: an arrival that carries them over is a release at cluster scope, and
    what arrives with less publishes only that tensor memory has been read."""
    text = source("e4m3_gemm_many.cu")
    barriers = dict(re.findall(r"(\w+)(?:\[\d\])? = \{?mapa_shared\(smem_u32\(&?(\w+)", text))
    plain = {barriers[name] for name in re.findall(r"mbar_arrive_cluster\((\w+)", text)}
    assert plain == {"tempty", "shared_free"}
    assert {barriers[name] for name in re.findall(r"mbar_arrive_release_cluster\((\w+)", text)} == {"sfull"}
    assert re.findall(r"mbar_wait\w*\(&sfull\[sb\]", text) == ["mbar_wait_cluster_warp(&sfull[sb]"]
    assert "mbarrier.arrive.release.cluster.shared::cluster.b64" in source("sm100_ptx.cuh")


def test_packing_walks_blocks_of_columns():
    """Up to 2^31 - 1024 columns in steps of up to 65535 blocks of 128: a column's number
    would pass 31 bits on its way past the last one, a block's does not."""
    start, bound, step = re.search(r"for \(int (\w+) = blockIdx\.y; \1 < (\w+); \1 \+= ([^)]+)\)", source("e4m3_rows.cu")).groups()
    assert (start, bound, step) == ("nb", "blocks", "gridDim.y")
    assert (2 ** 31 - 1024 + 127) // 128 + 65535 < 2 ** 31 <= 2 ** 31 - 1024 + 65535 * 128
