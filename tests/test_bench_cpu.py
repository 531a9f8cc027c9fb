"""The benchmark line's recorded figures against the sources they were taken on."""
import bench
from quantized_recurrent_state_lq_b200 import configs


def test_recorded_traffic_is_of_the_current_decode_sources():
    """bench.py reports the recorded DRAM bytes of the dominant decode kernel
    only while the code of the files that kernel is built from is the code the
    record was taken on: what other kernels need belongs in their own files."""
    got = bench.profile_traffic(configs.GDN_PREFIX_CACHE)
    assert got is not None and got > 0
