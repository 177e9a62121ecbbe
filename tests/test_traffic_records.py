"""The DRAM counters that bench.py reports beside its rooflines belong to the kernels as they are: a record
counts only while the sources it was taken on are unchanged."""
import bench


def test_records_of_the_measured_kernels_count():
    fine = bench.source_sha("fine_tc.cu", "sm100.cuh", "common.cuh")
    decode = bench.source_sha("decode_tc.cu", "mma_sync.cuh", "sm100.cuh", "common.cuh")
    assert bench.recorded_traffic("fine_tc_kernel", fine, "16k") is not None
    assert bench.recorded_traffic("decode_attn_tc_kernel", decode, "decode96k-b8") is not None
