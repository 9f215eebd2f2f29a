"""Host code of the launches, compiled by the host compiler alone with stand-ins for the runtime's calls."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def run_host(tmp_path, name):
    exe = str(tmp_path / name)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    os.path.join(HERE, "host", name + "_main.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "", r.stdout + r.stderr


def test_blocks_per_unit_follow_the_call(tmp_path):
    run_host(tmp_path, "launch_cache")


def test_choice_among_the_8_bit_products(tmp_path):
    run_host(tmp_path, "fp8_choice")
