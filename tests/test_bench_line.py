"""What bench.py prints, on the CPU: its traffic record is of the source that
is built, and its one line is short enough to be read whole."""
import json

import pytest

import bench

pytestmark = pytest.mark.cpu


def test_the_committed_traffic_record_is_of_the_current_source():
    traffic, how = bench.profiled_traffic()
    assert traffic is not None, how


def test_the_line_of_a_full_run_is_short_and_keeps_its_figures():
    """A run's tables as they come from 35 SM-budget rows, 21 message sizes and the rest, each row with its launch."""
    launch = ("allreduce_ldst dtype=bf16 op=sum p=16 n=117440512 schedule=ring variant=ldst vec=1 grid=152 block=512 smem=122880 "
              "sm_budget=152 counter=1 inplace=0")
    row = {"variant": "tma_bulkred", "sm_budget": 152, "ms": 18.343, "GBps": 1409.8, "GBps_per_SM": 102.44, "frac_of_hbm_peak": 0.0605,
           "launch": launch}
    arm = {"us": 14.975, "GBps": 6971.1, "frac_of_hbm_peak": 1.0394, "us_graph": 154.564}
    res = {"metric": "m", "value": 7061.25, "config": {"model": "c", "launch": launch}, "sm_budgets": [row] * 18, "sm_budgets_p8": [row] * 15,
           "sweep": [{"bytes_per_rank": 268435456, "rotating_sets": 64, "ring": arm, "allpairs": arm}] * 21, "e2e": {"value": 329.8},
           "fused_rmsnorm": {f"tokens_{i}": {"fused": arm, "allreduce_only": {"us": 1.0}, "launch": launch} for i in range(5)},
           "variants": {v: dict(arm, launch=launch) for v in ("ldst", "tma", "tma_bulkred", "ring_stepwise", "one_phase")}}
    line = bench.result_line(res)
    assert len(json.dumps(res)) > 13000 and len(line) < 12000 and "\n" not in line
    back = json.loads(line)
    assert back["value"] == 7061.25 and back["config"] == res["config"] and back["e2e"] == res["e2e"]
    assert [r["GBps"] for r in back["sm_budgets"]] == [1409.8] * 18 and back["sweep"] == res["sweep"]
    assert list(back) == list(res)
