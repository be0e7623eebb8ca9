"""Kernel attributes belong to a device: what the library sets once per device is set on each,
tried again after a failure, and no kernel sets one once per process.  (Host code; the
class has no CUDA call in it, so that a process with several devices can be played here.)"""
import glob
import os
import re
import shutil
import subprocess

import pytest

import gated_delta_rule_39_gb300 as package

CSRC = os.path.join(os.path.dirname(package.__file__), "csrc")

PROGRAM = r"""
#include "kda_per_device.h"
#include <cstdio>
int main() {
    static kda::OncePerDevice once;
    int calls[3] = {0, 0, 0}, answer = 0;
    auto at = [&](int dev) { return once(dev, [&] { ++calls[dev]; return answer; }); };
    int bad = 0;
    bad += at(0) != 0 || at(0) != 0 || calls[0] != 1;
    bad += at(1) != 0 || calls[1] != 1;      // another device: set there too
    answer = 7;
    bad += at(2) != 7 || calls[2] != 1;      // fails
    answer = 0;
    bad += at(2) != 0 || calls[2] != 2;      // and is tried again
    bad += at(2) != 0 || calls[2] != 2;
    std::printf("%d\n", bad);
    return bad;
}
"""


def test_every_device_is_set_once_and_failures_are_tried_again(tmp_path):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no g++")
    (tmp_path / "main.cpp").write_text(PROGRAM)
    subprocess.run([cc, "-std=c++17", "-I", CSRC, str(tmp_path / "main.cpp"), "-o", str(tmp_path / "main")], check=True)
    subprocess.run([str(tmp_path / "main")], check=True)


def test_no_result_of_a_cuda_call_is_kept_for_the_process():
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        with open(path) as f:
            found = re.search(r"static const cudaError_t", f.read())
        assert not found, path


@pytest.mark.gpu
def test_verify_in_the_largest_clusters():
    """16 CTAs per row, the size that needs the attribute."""
    torch = pytest.importorskip("torch")
    V = 50257
    target, noise = torch.rand(1, 1, V, device="cuda"), torch.rand(1, V, device="cuda") + 0.5
    accepted, tokens = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, 1, dtype=torch.int32, device="cuda")
    none = torch.empty(1, 0, dtype=torch.int32, device="cuda")
    package.kda_verify_drafts(target, None, none, none.float(), noise, accepted, tokens)
    assert tokens.item() == (target[0, 0] / noise[0]).argmax().item()
