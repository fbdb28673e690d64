"""CPU: gdn_pair_commit hands all of a sequence's state to its launcher at every
head count that its limits allow."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_states_past_32_bits(tmp_path):
    csrc = os.path.join(ROOT, "gated_deltanet_decode_amd", "csrc")
    cdir = os.path.join(ROOT, "tests", "c")
    exe = str(tmp_path / "gdn_commit_check")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-O1", "-g",
                    "-fno-omit-frame-pointer", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-I", os.path.join(ROOT, "include"), "-I", csrc, "-I", cdir,
                    os.path.join(csrc, "gdn_api.cpp"), os.path.join(csrc, "gdn_serve_api.cpp"),
                    os.path.join(cdir, "gdn_api_stubs.cpp"), os.path.join(cdir, "gdn_commit_check.cpp"),
                    "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "commit host check ok" in r.stdout
