"""Host-side checks of the prompt attention's sizes (tests/prompt_host_check.cu,
built with nvcc as a host-only program from the headers that the kernel
includes). No GPU needed."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    nvcc = shutil.which("nvcc") or ("/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else None)
    if nvcc is None:
        pytest.skip("nvcc not available")
    path = tmp_path_factory.mktemp("prompt_host")
    exe = str(path / "check")
    subprocess.run([nvcc, "-std=c++17", "-O2", "-o", exe, os.path.join(HERE, "prompt_host_check.cu")], check=True, capture_output=True,
                   cwd=str(path))

    def run(name):
        r = subprocess.run([exe, name], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
    return run


def test_copies_begin_on_boundaries(check):
    check("copies")


def test_the_largest_batches_are_dealt_to_the_threads(check):
    check("sequences")


def test_pieces_of_cut_units(check):
    check("pieces")
