"""The bench line's traffic figure (CPU)."""
import bench


def test_the_traffic_counters_belong_to_the_committed_kernel_sources():
    """The line reports measured FC1 traffic only while the grouped GEMM's sources are those that the
    counters were taken on; a change of them retakes profiles/fc1_swiglu_balanced_traffic.txt."""
    assert bench.measured_traffic("balanced") is not None
