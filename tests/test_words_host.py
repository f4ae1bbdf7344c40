"""The words that a recurrence's tiles hand on, folded on the CPU
(tests/words_check.cpp over varlen_depthwise_causal_amd/csrc/vdc_words.h): a fold
has the same bits wherever it begins, and a reader that gave up waiting has a NaN,
never a value that looks like a result."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_words_on_cpu(tmp_path):
    exe = str(tmp_path / "words_check")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror",
                    "-I", os.path.join(ROOT, "varlen_depthwise_causal_amd", "csrc"),
                    os.path.join(ROOT, "tests", "words_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout + out.stderr
    assert "words_check: ok" in out.stdout
