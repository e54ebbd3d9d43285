"""The recorded DRAM traffic of the decode and the prefill is of the kernels in
the tree (CPU only): a change of a source that they were captured on needs a
capture of its own, or a place in another file."""
import pytest

import bench


@pytest.mark.parametrize("config", ["opt13b-beam", "llama2-7b", "qwen3-prefix", "gqa-fp8", "gqa-int8"])
def test_the_recorded_decode_traffic_applies(config):
    assert bench.recorded_traffic(config) > 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "int8"])
def test_the_recorded_prefill_traffic_applies(cache):
    assert bench.recorded_traffic(cache, bench.PREFILL_TRAFFIC_FILE, bench.PREFILL_SOURCES) > 0
