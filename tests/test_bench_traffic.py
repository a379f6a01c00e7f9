"""bench.py's DRAM traffic figure belongs to the GEMM's sources as they stand
(it is reported as null for others)."""
import bench


def test_the_captured_traffic_is_of_these_sources():
    assert bench.gemm_traffic(bench.GEMM_TRAFFIC["workload"]) == 1844060850
    assert bench.gemm_traffic("another") is None
