"""The packed and paged calls on the bounds-checked build: no check fires, and
every output, state and pool equals the production build's bit for bit."""
import os
import subprocess
import sys

import numpy as np
import pytest

from int4_quantized_attention_b200 import api, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def run_worker(tmp_path, library):
    out = str(tmp_path / f"{library}.npz")
    r = subprocess.run([sys.executable, os.path.join(HERE, "serve_bounds_worker.py"), out],
                       env=dict(os.environ, RA_LIBRARY=library), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return dict(np.load(out))


def test_bounds_build_reports_nothing_and_matches(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    checked, plain = run_worker(tmp_path, "bounds"), run_worker(tmp_path, "production")
    assert set(checked) == set(plain)
    for key, val in plain.items():
        if key.endswith("status"):
            assert int(val) == int(checked[key]) == api.RA_OK, key
        else:
            assert np.array_equal(checked[key], val), key
