"""The committed DRAM traffic of the single-pass quantizer belongs to the source that is here: bench.py reports no
traffic otherwise."""
import bench


def test_traffic_record_is_current():
    assert bench._traffic_record() is not None, "capture it again (see profiles/nvfp4_quant_gate_up_fullsize_traffic.txt)"
    split = bench.ncu_traffic_split()
    assert bench.ncu_traffic_per_launch() == split["traffic_read"] + split["traffic_write"]
    # one pass over the 3.2 GB of input; the outputs may still lie in L2 when the kernel ends
    assert 0.98 < split["traffic_read"] / (512 * 1536 * 2048 * 2) < 1.05
