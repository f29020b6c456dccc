"""The lookup of the tensor-map encoder by many host threads at once, in a process
of its own, without a GPU (tests/encode_threads.cu)."""
import os
import subprocess

from speculative_decoding_verification_vocab_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_first_calls_of_many_threads(tmp_path):
    program = str(tmp_path / "encode_threads")
    built = subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-I", _build.INCLUDE, "-I", _build.CSRC, "-o", program,
                            os.path.join(HERE, "encode_threads.cu")], capture_output=True, text=True)
    assert built.returncode == 0, built.stderr[-2000:]
    r = subprocess.run([program], capture_output=True, text=True, timeout=60)
    assert (r.returncode, r.stdout) == (0, "0 wrong, 1 queries\n"), r.stderr
