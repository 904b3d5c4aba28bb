"""The host side of the scoring operators, the RMS norm and the gradient norm (score_abi.cpp, train_abi.cpp) under
AddressSanitizer and UndefinedBehaviorSanitizer, driven by native/score_abi_stub.cpp: built host-only, launches are looked
at instead of made, and no GPU is visible."""
import os

import pytest

shared = pytest.importorskip("test_sanitizers")    # its runner and flags
ENV, ROOT, SAN_HIP = shared.ENV, shared.ROOT, shared.SAN_HIP
need, rl, rl_build, run = shared.need, shared.rl, shared.rl_build, shared.run


def test_host_scoring_abi_under_sanitizers(tmp_path):
    hipcc = need("hipcc")
    lib = rl.library_path()
    if not os.path.exists(lib):
        rl_build.build()
    exe = tmp_path / "score_abi_stub"
    rc, out = run([hipcc, "--offload-host-only", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", *SAN_HIP,
                   "-I", os.path.join(ROOT, "include"), "-I", rl_build.CSRC,
                   os.path.join(rl_build.CSRC, "score_abi.cpp"), os.path.join(rl_build.CSRC, "train_abi.cpp"),
                   os.path.join(ROOT, "tests", "native", "score_abi_stub.cpp"),
                   "-L", os.path.dirname(lib), "-lrl_post_loss", "-Wl,-rpath," + os.path.dirname(lib), "-o", str(exe)])
    assert rc == 0, out
    env = dict(ENV, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")
    rc, out = run([str(exe)], env=env)
    assert rc == 0 and out.startswith("ok "), out
