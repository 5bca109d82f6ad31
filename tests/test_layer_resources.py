"""Registers, scratch and LDS of the convolution's, the scan's and the norm's kernels, from the compiler's own resource report
(host-side compilation for gfx950; no GPU).  Vector issue binds the scan, so the waves that a SIMD holds count: three and more
forward; backward three with 16 states of 16-bit rows, two otherwise, and one with 32 states of binary32 rows, whose
registers do not fit twice.  Only the norm's gradient of rows above 16,384 columns spills."""
import re
import shutil

import pytest

from quantized_delta_rule_amd import build

from test_kernel_resources import HIPCC

pytestmark = pytest.mark.skipif(not shutil.which(HIPCC), reason="hipcc not available")
F32 = 0


@pytest.fixture(scope="module")
def resources():
    """{(kernel, its template's numbers): report}"""
    out = {}
    for name, r in build.kernel_resources(build.LAYER_SOURCES).items():
        m = re.match(r"_ZN5stepq12_GLOBAL__N_1(\d+)(k_\w+)$", name)
        kernel, rest = m.group(2)[:int(m.group(1))], m.group(2)[int(m.group(1)):]
        numbers = re.match(r"I((?:Li\d+E)+)E", rest)
        out[kernel, tuple(map(int, re.findall(r"\d+", numbers.group(1) if numbers else "")))] = r
    return out


def test_every_kernel_is_reported(resources):
    count = {}
    for kernel, _ in resources:
        count[kernel] = count.get(kernel, 0) + 1
    # types x widths, x row lengths, x states; passes 0 to 2 of the forward scan's states and 1 and 3 of the gradient's
    assert count == {"k_conv": 9, "k_conv_grad": 9, "k_norm": 27, "k_norm_grad": 27, "k_scan_tokens": 12, "k_scan_run": 51,
                     "k_scan_back": 36, "k_scan_bc": 3, "k_sum": 1}


def test_no_spills(resources):
    for (kernel, numbers), r in resources.items():
        if kernel == "k_norm_grad" and numbers[1:] == (1024, 4):
            continue
        assert r["ScratchSize"] == 0 and r["VGPRs Spill"] == 0 and r["SGPRs Spill"] == 0, (kernel, numbers, r)


def test_waves_of_the_scan(resources):
    for (kernel, numbers), r in resources.items():
        if kernel == "k_scan_run":
            assert r["Occupancy"] >= 3, (numbers, r)
        elif kernel == "k_scan_back":
            dt, ns, nw, what = numbers
            least = 5 if what == 1 else 3 if dt != F32 and (ns, nw) == (2, 4) else 1 if dt == F32 and (ns, nw) == (4, 4) else 2
            assert r["Occupancy"] >= least and r["LDS Size"] <= 163840 // 2 * (2 if nw == 8 else 1), (numbers, r)
        elif kernel == "k_scan_tokens":
            assert r["Occupancy"] >= 7, (numbers, r)


def test_waves_of_the_others(resources):
    """Bound by memory: enough rows in flight."""
    for (kernel, numbers), r in resources.items():
        if kernel in ("k_norm", "k_sum", "k_scan_bc"):
            assert r["Occupancy"] >= 4, (kernel, numbers, r)
        elif kernel in ("k_conv", "k_conv_grad"):
            assert r["Occupancy"] >= 3, (kernel, numbers, r)
