"""The benchmark reports measured DRAM traffic only for the source it was captured
on, so a changed kernel source without a new capture loses the figures without a
sign: every stored figure is of the sources as they are."""
import bench


def test_stored_traffic_is_of_the_current_sources():
    assert {h for h, _ in bench.TRAFFIC.values()} == {bench._source_hash("gqa_decode.cu")}
    assert {h for h, _ in bench.PREFILL_TRAFFIC.values()} == {bench._source_hash("prefill.cu")}
    assert {w for w, _ in bench.TRAFFIC} == {bench.DEFAULT_WORKLOAD, *bench.SUB_WORKLOADS}
