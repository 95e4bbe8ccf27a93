"""bench.py refuses options that name no workload, rather than timing another one."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("options, word", [(["--int8"], "--infer"), (["--infer", "--int8", "--static"], "--int8"),
                                           (["--infer", "--repair"], "--repair"), (["--repair", "--int8"], "--infer")])
def test_options_that_name_no_workload(options, word):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), *options], capture_output=True, text=True, timeout=60)
    assert r.returncode == 2 and word in r.stderr and not r.stdout


@pytest.mark.parametrize("options, word", [(["--int4"], "--infer"), (["--infer", "--int4", "--int8"], "--int8"),
                                           (["--infer", "--int4", "--static"], "--int4"), (["--repair", "--int4"], "--infer")])
def test_options_of_4_bits_that_name_no_workload(options, word):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), *options], capture_output=True, text=True, timeout=60)
    assert r.returncode == 2 and word in r.stderr and not r.stdout
