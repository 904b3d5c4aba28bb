"""The host side of the scoring operators, the RMS norm and the gradient norm against a HIP runtime that the test makes up
(native/score_abi_stub.cpp): extreme arguments, and the launches that the others make.  No GPU takes part."""
import os
import re
import shutil
import subprocess

import pytest

import rl_post_loss_amd as rl
from rl_post_loss_amd import build as rl_build

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native")


def test_against_a_runtime_of_its_own(tmp_path):
    hipcc = shutil.which("hipcc")
    if hipcc is None:
        pytest.skip("needs hipcc")
    lib = rl.library_path()
    if not os.path.exists(lib):
        rl_build.build()
    exe = str(tmp_path / "score_abi_stub")
    r = subprocess.run([hipcc, "--offload-host-only", "-std=c++17", "-O1", "-I", rl_build.INCLUDE, "-I", rl_build.CSRC,
                        os.path.join(rl_build.CSRC, "score_abi.cpp"), os.path.join(rl_build.CSRC, "train_abi.cpp"),
                        os.path.join(HERE, "score_abi_stub.cpp"),
                        "-L", os.path.dirname(lib), "-lrl_post_loss", "-Wl,-rpath," + os.path.dirname(lib), "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1"))
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr


def test_the_header_states_the_bounds_that_the_code_has():
    """The bounds that native/score_abi_stub.cpp finds in the code."""
    text = re.sub(r"\s*\n \*\s*", " ", open(os.path.join(rl_build.INCLUDE, "rl_post_loss.h")).read())
    for bound in ("fewer than 2^24 tiles of 64 rows by 64 entries", "2^20", "2^22", "2^31 - 65536"):
        assert bound in text, bound
