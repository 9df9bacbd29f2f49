"""The DRAM counters that bench.py reports belong to the kernels as they are (CPU only)."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("src,kernel,workload", [("decode.cu", "decode_fused", "ling_t1"), ("umma.cu", "routed_gateup", "prefill_t4096"),
                                                 ("tcdense.cu", "combine", "prefill_t4096"), ("lmhead.cu", "lm_gemv", "lmhead_t1")])
def test_counters_of_the_current_source(src, kernel, workload):
    spec = importlib.util.spec_from_file_location("bench_mod", os.path.join(ROOT, "bench.py"))
    bench = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(bench)
    path = os.path.join(ROOT, "mxfp4_expert_gb300", "csrc", src)
    assert bench.profiled_traffic(path, kernel, workload) is not None
