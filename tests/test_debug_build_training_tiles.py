"""The bounds-checked build's checks of the expert training calls in tiles of 256 x 256 and 128 x 128
(tests/debug_child_training.py takes those of 64 x 64): a child process on the checked library runs clean
inputs, gaps between segments among them, with no flag raised, then out-of-range row segments and sorted
indices, each kept from use and named by its flag."""
import os
import subprocess
import sys

import pytest
import torch

from conftest import ROOT
from test_debug_build import _env


@pytest.mark.gpu
@pytest.mark.timeout(400)
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
def test_checked_build_on_gpu():
    print("[debug build] child process on the checked library", flush=True)
    r = subprocess.run([sys.executable, "-u", os.path.join(ROOT, "tests", "debug_child_training_tiles.py")],
                       cwd=ROOT, env=_env(), capture_output=True, text=True, timeout=360)
    print(r.stdout[-6000:], r.stderr[-3000:], flush=True)
    assert r.returncode == 0
    assert "DEBUG CHILD OK" in r.stdout
