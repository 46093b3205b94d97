"""Rules that the sources of the 8-bit projections keep, read from the files."""
import glob
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


def test_ctas_that_wait_for_others_find_tensor_memory_where_they_find_shared_memory():
    """Tensor memory is waited for without a limit, and the CTAs of a cluster wait for one
    another: whatever CTAs of the two products for few rows share an SM (228 KB, 1 KB each for
    itself), their 32-bit columns are at most its 512."""
    text, skinny = source("e4m3_gemm_few.cu"), source("gemm_skinny.cu")
    ctas = []
    forms = {tuple(map(int, f)) for f in re.findall(r"return go<(\d+), (\d+), (\d+)>", text)}
    assert len(forms) == 7
    for nt, mats, cps in forms:
        for one, per_sm in ((True, 2), (False, cps)):
            if one and re.search(r"if constexpr \(MATS == 1 \|\| NT < 64\)", text) and mats == 2 and nt == 64:
                continue                                # (not there)
            stage = mats * 128 * 128 + nt * 128
            inbox = 32 * 128 * 4 if one and mats == 1 and nt <= 32 else 0
            stages = min(12, ((110 if per_sm == 2 else 220) * 1024 - inbox) // stage)
            smem = stages * stage + inbox + 512 + 1024
            columns = mats * nt * (1 if one else 2) + (4 if one else 8) * (4 * mats + 4)
            ctas.append((smem, next(c for c in (128, 256, 512) if c >= columns)))
    assert re.search(r"TMEM_COLS = NT <= 32 \? 32 : 64", skinny)
    for nt, stages in ((16, 5), (32, 5), (48, 4), (64, 4), (16, 3), (32, 3)):
        ctas.append((stages * (16384 + nt * 128) + 128 + 256 + 2048 + 16 + 1024, 32 if nt <= 32 else 64))

    def fill(room, columns, first):
        assert columns <= 512, columns
        for i in range(first, len(ctas)):
            if ctas[i][0] + 1024 <= room:
                fill(room - ctas[i][0] - 1024, columns + ctas[i][1], i)

    fill(228 * 1024, 0, 0)


def test_dependents_are_let_in_once_tensor_memory_is_there():
    """The allocation waits for CTAs of the SM; one of the next launch among them would be
    waiting for this one to end."""
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = code(path)
        for kernel in re.split(r"__global__", text)[1:]:
            took = [m.start() for m in re.finditer(r"\btmem_alloc(?:_pair)?\(", kernel)]
            let = [m.start() for m in re.finditer(r"\bpdl_trigger\(\)", kernel)]
            if took and let:
                seen += 1
                # (by the warp that allocates, which goes on once it has it)
                assert min(let) > max(took), os.path.basename(path)
                assert re.match(r"pdl_trigger\(\);\s*\}\s*tc_fence_before\(\);", kernel[min(let):]), os.path.basename(path)
    assert seen == 4


def test_waits_with_a_limit_begin_when_the_kernel_ahead_has_ended():
    """A CTA may be resident long before: no warp counts that time against the two seconds
    after which a wait is given up."""
    for name in ("e4m3_gemm_few.cu", "e4m3_gemm_many.cu", "gemm_skinny.cu"):
        text = source(name)
        roles = re.split(r"\n  (?:if|\} else if) \(warp (?:==|>=) \d+\) \{|\n  \} else \{", text[text.index("uint32_t tmem = *tmem_slot"):])[1:]
        roles = [r for r in roles if "mbar_wait" in r or "mbar_try_wait" in r][:4]
        assert len(roles) >= 3
        for r in roles[:3]:
            first = re.search(r"mbar_(?:try_)?wait\w*\(", r).start()
            # (the loads of the few-rows kernels wait for a stage only once all have been filled and released)
            assert "pdl_wait()" in r[:first] or "release();" in r, name
