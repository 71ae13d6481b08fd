"""The benchmark's stored counter readings belong to the scan sources as they are."""
import json
import os

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_stored_traffic_is_of_the_present_scan_sources():
    """A change to the scan's sources retires the readings and the benchmark reports
    none: take the counters again, or, where the scan kernels' device code is the
    same instruction for instruction, enter the sources' new digest."""
    for key in json.load(open(os.path.join(ROOT, "profiles", "traffic.json"))):
        assert bench.stored_traffic(*key.split(":")) is not None, key


def test_scan_sources_hold_no_other_operators():
    for name in bench.SCAN_SOURCES:
        path = os.path.join(ROOT, "approximate_nearest_neighbour_amd", "csrc", name)
        text = open(path).read()
        assert "mx4" not in text and "route_" not in text, name
