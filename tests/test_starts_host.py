"""The search for the documents around one token, run on the CPU
(tests/starts_check.cpp over varlen_depthwise_causal_amd/csrc/vdc_search.h): the
documents that end and start there, past any number of empty ones, in at most 64
probes, none of them outside cu_seqlens whatever it holds."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_documents_around_a_token_on_cpu(tmp_path):
    exe = str(tmp_path / "starts_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror",
                    "-I", os.path.join(ROOT, "varlen_depthwise_causal_amd", "csrc"),
                    os.path.join(ROOT, "tests", "starts_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout + out.stderr
    assert "starts_check: ok" in out.stdout
