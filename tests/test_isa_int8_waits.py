"""The int8 products wait only as designed (CPU: cross-compiled gfx950 assembly, no
GPU): from the first load to LDS up to the end of the stage loop a kernel holds
the ring's waits and none that drains it (the compiler adds one wherever it
believes that a read from LDS may see a load in flight)."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "moe_grouped_block_mx_amd", "csrc", "gemm_int8.hip")


def _hipcc():
    h = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    return h if os.path.exists(h) else None


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if _hipcc() is None:
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("isa") / "int8.s"
    cmd = [_hipcc(), "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", f"-I{os.path.join(ROOT, 'include')}", "-S", "--cuda-device-only", SRC, "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    found, name = {}, None
    for line in out.read_text().splitlines():
        m = re.match(r"_ZN4mxgg\S*?(grouped|split|few)_int8_kernelI(\S*?)EEv", line)
        if m and line.split(";")[0].strip().endswith(":"):
            name = (m.group(1), tuple(int(v) for v in re.findall(r"Li(\d+)E", m.group(2) + "E")))
            found[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name:
            found[name].append(line)
    return found


def waits(lines):
    return [int(m.group(1)) for line in lines if (m := re.search(r"s_waitcnt .*vmcnt\((\d+)\)", line))]


def region(kind, lines):
    """From the first load to LDS to the last MFMA; in a few-rows kernel, whose
    waves join their sums behind it, to the barrier before they do."""
    first = next(i for i, line in enumerate(lines) if re.search(r"load_dword\S* .* lds", line))
    last = max(i for i, line in enumerate(lines) if "v_mfma" in line)
    end = next(i for i in range(last, len(lines)) if "s_barrier" in lines[i]) if kind == "few" else last
    return lines[first:end]


def test_every_kernel_is_there(kernels):
    assert {k[0] for k in kernels} == {"grouped", "split", "few"} and len(kernels) == 9


def test_ring_waits(kernels):
    for (kind, args), lines in kernels.items():
        got = waits(region(kind, lines))
        if kind == "few":
            nf, mf = args
            slots = {2: 4, 3: 3, 4: 4, 6: 3, 8: 2}[nf + mf]
            # the loop's wait; the drain behind it
            assert got == [(slots - 1) * (nf + mf), 0], (kind, args, got)
        else:
            fn, fm, ku, slots = args
            tn, tm = 32 * fn, (64 if kind == "grouped" else 32) * fm
            ahead = (slots - 2) * (tn + tm) * 64 * ku // 8192
            assert got and set(got) == {ahead}, (kind, args, got)


def test_no_register_is_spilled(kernels):
    for name, lines in kernels.items():
        assert not any("scratch_" in line for line in lines), name
