"""The build's reading of the compiler's remarks: a kernel that spills registers no one has allowed for is an
error."""
from post_weight_quantization_amd import build

REMARKS = """\
a.hip:9:1: remark: Function Name: _ZN4gptq21attention_tile_kernelILi0ELi8EEEvNS_8AttnArgsE [-Rpass-analysis=kernel-resource-usage]
a.hip:9:1: remark:     VGPRs: 256 [-Rpass-analysis=kernel-resource-usage]
a.hip:9:1: remark:     SGPRs Spill: 7 [-Rpass-analysis=kernel-resource-usage]
a.hip:9:1: remark:     VGPRs Spill: 28 [-Rpass-analysis=kernel-resource-usage]
a.hip:20:1: remark: Function Name: _ZN4gptq21attention_rows_kernelILi1ELi4EEEvNS_8AttnArgsE [-Rpass-analysis=kernel-resource-usage]
a.hip:20:1: remark:     VGPRs Spill: 0 [-Rpass-analysis=kernel-resource-usage]
"""


def test_stated_spills_pass():
    found = build.spills(REMARKS)
    assert found == {"_ZN4gptq21attention_tile_kernelILi0ELi8EEEvNS_8AttnArgsE": 28}
    assert build.too_many(found) == []


def test_others_do_not():
    assert len(build.too_many(build.spills(REMARKS.replace("Spill: 28", "Spill: 29")))) == 1
    assert len(build.too_many(build.spills(REMARKS.replace("VGPRs Spill: 0", "VGPRs Spill: 9")))) == 1


def test_the_build_asks_for_the_remarks():
    assert "-Rpass-analysis=kernel-resource-usage" in build.FLAGS
