"""The build rejects kernels that registers leave fewer waves than their plan counts on (CPU
only)."""
from quantized_gemm_rtn_amd.build import LEAST_WAVES, too_few_waves


def test_wave_guard_reads_resource_remarks():
    remarks = "\n".join([
        "a.hip:1:1: remark: Function Name: _Z7kernelAv [-Rpass-analysis=kernel-resource-usage]",
        "a.hip:1:1: remark:     TotalVGPRs: 251 [-Rpass-analysis=kernel-resource-usage]",
        "a.hip:1:1: remark:     Occupancy [waves/SIMD]: 2 [-Rpass-analysis=kernel-resource-usage]",
        "a.hip:9:1: remark: Function Name: _Z7kernelBv [-Rpass-analysis=kernel-resource-usage]",
        "a.hip:9:1: remark:     Occupancy [waves/SIMD]: 1 [-Rpass-analysis=kernel-resource-usage]",
    ])
    assert too_few_waves(remarks, {"kernelA": 2}) == {}
    assert too_few_waves(remarks, {"kernelA": 2, "kernelB": 2}) == {"_Z7kernelBv": 1}
    assert too_few_waves(remarks, {"kernelC": 1}) == {"kernelC": None}
    assert too_few_waves("", {}) == {}
    assert LEAST_WAVES["kv4_tile.hip"] == {"kv4_tile_kernel": 2}
