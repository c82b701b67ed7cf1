"""The training operators under their checked build (libqt2_train_checked.so: every kernel store is
checked against its array), and their first calls inside a graph capture."""
import os
import subprocess
import sys

import pytest

from nvfp4_quantized_b200 import build as qbuild
from nvfp4_quantized_b200 import qt2_train as tr

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_suites_pass_under_the_checked_build():
    qbuild.build(checked=True)
    qbuild.build_train(checked=True)
    env = dict(os.environ, QT2_LIBRARY="checked")
    files = ["tests/test_gpu_norm.py", "tests/test_gpu_xent.py", "tests/test_gpu_grad.py", "tests/test_gpu_train_step.py"]
    r = subprocess.run([sys.executable, "-m", "pytest", *files, "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1500)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert not tr.qt2_train_build_checked()


FIRST = """
import torch
from nvfp4_quantized_b200 import qt2, qt2_train as tr
from tests.test_gpu_train_step import Step
assert {checked} == tr.qt2_train_build_checked()
s = Step(1)
torch.cuda.synchronize()
graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(graph, stream=side):
    s.run()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in s.outputs()]
s.run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, s.outputs()))
assert qt2.qt2_device_status() == 0 and tr.qt2_train_device_status() == 0
print("ok")
"""


def test_first_calls_of_a_process_in_a_capture():
    r = subprocess.run([sys.executable, "-c", FIRST.format(checked=False)], cwd=ROOT, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
