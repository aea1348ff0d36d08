"""The committed counter summaries that bench.py reads belong to the committed kernels."""
import bench


def test_fold_traffic_belongs_to_the_sources():
    """The record is tied to the fold's sources by their hash; after a change to them the counters are taken again."""
    traffic = bench.recorded_traffic()
    assert traffic is not None, "profiles/fold_update_traffic_n17408.md is of other sources: take its counters again"
    # A launch updates part of one matrix of 17408 columns: more than a panel of 512 rows, less than all of it
    # read twice and written once.
    assert 512 * 17408 * 4 < traffic < 3 * 17408 ** 2 * 4


def test_sweep_traffic_is_read():
    assert bench.recorded_sweep_dram_bytes() > 1e9
