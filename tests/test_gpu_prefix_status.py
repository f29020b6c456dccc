"""The status of a prefix attention in which a wait ran out, on a made-up workspace
(tests/prefix_status.cu): nothing waits here."""
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

sv = pytest.importorskip("speculative_decoding_verification_vocab_gb300")
from speculative_decoding_verification_vocab_gb300 import _build  # noqa: E402

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")
def test_a_wait_that_ran_out_is_told_to_every_sequence_it_concerns(tmp_path):
    program = str(tmp_path / "prefix_status")
    built = subprocess.run([_build.nvcc(), *_build.ARCH, "-O1", "-std=c++17", "-I", _build.INCLUDE, "-I", _build.CSRC, "-o", program,
                            os.path.join(HERE, "prefix_status.cu"), os.path.join(_build.CSRC, "runtime.cu")],
                           capture_output=True, text=True)
    assert built.returncode == 0, built.stderr[-3000:]
    r = subprocess.run([program], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
