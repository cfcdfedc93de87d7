"""The HBM traffic that bench.py reports belongs to the kernel as it is: the
record's digest is the sources' (a change that leaves the reroute's machine
code alone renews the digest, any other one the counters)."""
import bench


def test_recorded_traffic_belongs_to_the_sources():
    assert bench.measured_traffic() is not None
