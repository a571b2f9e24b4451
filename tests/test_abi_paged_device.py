"""Calls that pass validation without a GPU behind them: what they return, and
that none of them is made with invented addresses where a GPU is present."""
import os
import subprocess
import sys

import pytest
import torch

import conftest
import test_abi_paged as host

OK, NO_DEVICE = host.OK, host.NO_DEVICE
lib = host.lib

def test_invented_addresses_stay_off_a_gpu(lib, tmp_path):
    # a run of its own in which a GPU seems to be present (it has none, whatever the
    # machine has) and an entry point that is reached fails
    (tmp_path / "seems_gpu.py").write_text(
        "import torch\n"
        "torch.cuda.is_available = lambda: True\n"
        "from sequence_depth_attention_gb300 import binding\n"
        "lib = binding.load()\n"
        "def reached(*args):\n"
        "    raise AssertionError('an entry point is reached')\n"
        "for name in ('moda_fwd', 'moda_kv_append'):\n"
        "    lib.__dict__[name] = reached\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=os.pathsep.join((str(tmp_path), root)))
    tests = sorted(os.path.join(root, "tests", t) for t in conftest.INVENTED_ADDRESSES)
    r = subprocess.run([sys.executable, "-m", "pytest", "-p", "seems_gpu", "-q", "-p", "no:cacheprovider", *tests],
                       env=env, cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and f"{len(tests)} skipped" in r.stdout, r.stdout + r.stderr


def test_append_of_no_tokens(lib):
    assert host.append(lib, N=0, k=None, v=None, seq=None) == OK


def test_calls_that_pass_validation_end_at_the_device(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    # no queries, no rotation, no k_out, strides of a single token unused
    assert host.append(lib, q=None, qo=None, Hq=0, ko=None, rope=None, rows=0, rot=0, N=1, ks=3,
                       vs=5) == NO_DEVICE
    assert host.append(lib) == NO_DEVICE
    assert host.gather(lib) == NO_DEVICE
    assert host.decode(lib) == NO_DEVICE
    assert host.decode(lib, kd=None, vd=None, L=0, lse=None) == NO_DEVICE
