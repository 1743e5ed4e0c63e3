"""Failure detection of the large low-rank tiles: bounded waits that run out.

A warp whose wait runs out stops fetching, multiplying or storing, meets its
cluster's barriers all the same, and leaves only when what it has under way is
done; the plan's error word tells the host.  A test build with waits of ~1 ms
withholds the copies of a tile from some point on, so nothing that is waited for
is in flight (operators_runout_probe.py, in a subprocess of its own).
"""
import json
import os
import subprocess
import sys
import tempfile

import pytest

from ragged_blocked_kv_raggedbatch_gb300 import build as B

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_withheld_copies_are_reported_and_the_next_call_is_right():
    out_dir = os.path.join(tempfile.gettempdir(), "ds_ragged_wait_runout_build")
    lib = B.build(out_dir=out_dir, extra_flags="-DDSR_TEST_WAIT_RUNOUT")
    r = subprocess.run([sys.executable, os.path.join(HERE, "operators_runout_probe.py"), lib],
                       capture_output=True, text=True, timeout=600)
    lines = [x for x in r.stdout.splitlines() if x.startswith("{")]
    assert lines, r.stdout[-2000:] + r.stderr[-3000:]
    res = json.loads(lines[-1])
    assert r.returncode == 0 and res["ok"], [x for x in res["runs"] if x["error"] != 4 or x["after"] or not x["right"]]
