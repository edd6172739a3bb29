"""Race check of the gated products' LDS pipelines: the race-check build, whose
LDS-DMA copies first poison what they will write (see test_poison_lds_gpu),
must give bitwise the released build's bytes for every tile kind and pipeline of
gated_poison_cases.  It runs in a child process, as the library is chosen when
a process first loads it.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

from .gpu_util import log, torch
from .test_poison_lds_gpu import HERE, POISON_LIB

pytestmark = pytest.mark.gpu


def test_poison_build_matches_released_build(tmp_path):
    t = torch()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    assert os.path.exists(POISON_LIB), "race-check build missing: run __graft_entry__.build()"
    from . import gated_poison_cases
    ref = gated_poison_cases.run_cases()
    out = str(tmp_path / "poison.npz")
    r = subprocess.run([sys.executable, os.path.join(HERE, "gated_poison_cases.py"), out],
                       capture_output=True, text=True, env=dict(os.environ, FP8BLK_LIB=POISON_LIB),
                       timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    got = np.load(out)
    assert sorted(got.files) == sorted(ref)
    for name in sorted(ref):
        nbad = int((got[name] != ref[name]).sum())
        log(f"  {name}: {ref[name].size} bytes, {nbad} differ")
        assert nbad == 0, name
