"""Long lists, many tokens and forks on the bounds-checked build: no check of
the page operations or of the attention's rows, parts and table columns fires,
and every output, state and pool equals the production build's bit for bit."""
import os
import subprocess
import sys

import numpy as np
import pytest

from int4_quantized_attention_b200 import api, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_wide_lists_on_the_bounds_build(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    got = {}
    for library in ("bounds", "production"):
        out = str(tmp_path / f"{library}.npz")
        r = subprocess.run([sys.executable, os.path.join(HERE, "serve_bounds_wide_worker.py"), out],
                           env=dict(os.environ, RA_LIBRARY=library), capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
        got[library] = dict(np.load(out))
    assert set(got["bounds"]) == set(got["production"])
    for key, val in got["production"].items():
        if key.endswith("status"):
            assert int(val) == int(got["bounds"][key]) == api.RA_OK, key
        else:
            assert np.array_equal(got["bounds"][key], val), key
