"""The split of a decode whose warps run alone, from lengths to subtiles, on the host."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_place_replay(tmp_path):
    exe = tmp_path / "warp_place_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "paged_kv_cache_47_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "warp_place_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "OK", r.stdout
