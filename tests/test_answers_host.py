"""The table of a device's answers (how many clusters it holds at once): each device
answers for itself, and a failed query is not kept."""
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "state_space_model_chunked_gb300", "csrc")


def test_answers_are_kept_by_device_and_failures_are_not(tmp_path):
    out = str(tmp_path / "answers_check")
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, os.path.join(HERE, "answers_check.cpp"), "-o", out],
                   check=True)
    r = subprocess.run([out], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_the_product_asks_through_the_table():
    text = open(os.path.join(CSRC, "linear_tc.cu")).read()
    body = text[text.index("int clusters_at_once("):]
    body = body[:body.index("\n}\n")]
    assert "SsdAnswers" in body and "cudaGetDevice" in body and "std::atomic" not in text
