"""The bounds-checked debug build on what is most likely to leave a buffer:
offsets, row indices and slots that are not valid, the expert layer as a whole,
and calls back to back on shared buffers."""
import os
import subprocess
import sys

import pytest

import nvfp4_w4a4_quantized_10_b200 as nv

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = ["tests/test_gpu_grouped.py::test_bad_offsets_are_reported_and_nothing_is_written",
         "tests/test_gpu_grouped.py::test_bad_row_index_is_reported_and_quantized_as_zeros",
         "tests/test_gpu_expert_layer.py::test_layer", "tests/test_gpu_expert_layer.py::test_layer_as_a_graph_on_other_inputs",
         "tests/test_gpu_expert_layer_streams.py", "tests/test_gpu_back_to_back.py", "tests/test_gpu_block_norm_slots.py",
         "tests/test_gpu_grouped_swiglu.py", "tests/test_gpu_route_infinite.py", "tests/test_gpu_scale_borders.py"]


def test_these_pass_on_the_debug_build():
    if nv.DEBUG_BOUNDS:
        pytest.skip("this is the debug build")
    env = dict(os.environ, NVFP4_DEBUG_BOUNDS="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider"] + TESTS,
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1500)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert "skipped" not in r.stdout and "deselected" not in r.stdout, r.stdout[-500:]
