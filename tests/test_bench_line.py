"""What bench.py prints, on the CPU: its traffic record is of the source that
is built, and its one line is short enough to be read whole."""
import json

import pytest

import bench

pytestmark = pytest.mark.cpu


def test_the_committed_traffic_record_is_of_the_current_source():
    traffic, how = bench.profiled_traffic()
    assert traffic is not None, how
