"""bench.py's serving case: its lengths, and (on a GPU) its line."""
import json
import os
import subprocess
import sys

import pytest

import bench


def test_serve_lengths_span_half_to_all_of_the_stated_context():
    assert bench.serve_lengths(1, 1000) == [1000]        # one request: of the stated length
    assert bench.serve_lengths(2, 1001) == [1001, 500]
    n = bench.serve_lengths(32, 8192)
    assert len(n) == 32 and n[0] == max(n) == 8192 and n[-1] == min(n) == 4096 and len(set(n)) == 32


@pytest.mark.gpu
def test_serve_line_states_its_tokens_and_layout():
    root = os.path.dirname(os.path.abspath(bench.__file__))
    cmd = [sys.executable, "bench.py", "--case", "serve", "--shape", "1,8,100,64", "--nq", "2", "--steps", "3", "--warmup", "3"]
    r = subprocess.run(cmd, cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    line = json.loads(r.stdout.strip().splitlines()[-1])
    assert line["cached_tokens"] == 100 and line["inputs"] == "token-major projection" and line["ms_per_step"] > 0
