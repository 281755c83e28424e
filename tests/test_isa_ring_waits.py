"""The few-token expert layer's products wait only as designed (CPU:
cross-compiled gfx950 assembly, no GPU). A wave's ring has SLOTS - 2 pieces in
flight behind the one it waits for, each of RT + 1 + XN loads to LDS; the
compiler adds a full drain wherever it believes that an LDS read may see a load
in flight (reads through HIP's uint4 struct are enough for that), and such a
drain in the loop stalls every piece. From its first load to LDS to the barrier
behind the loop a kernel must hold exactly the ring's wait and, in the second
product (whose loop is its only one), the drain at the loop's end."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "moe_grouped_block_mx_amd", "csrc", "moe_layer.hip")


def _hipcc():
    h = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    return h if os.path.exists(h) else None


def _cut(name):
    """(RT, XN, SLOTS) of a kernel from its template arguments (UpCut, DownCut)."""
    up = re.search(r"moe_up_kernelILNS_9MoeFormatE\dELi(\d)ELb[01]E", name)
    if up:
        xn = int(up.group(1))
        return 2 if xn == 1 else 4, xn, {1: 5, 2: 5, 3: 4}[xn]
    rt, xn, many = map(int, re.search(r"moe_down_kernelILNS_9MoeFormatE\dELi(\d)ELi(\d)ELb[01]ELb([01])E", name).groups())
    slots = {4: (5 if xn == 1 else 4) - many, 1: 4}[rt]
    return rt, xn, slots


@pytest.mark.skipif(_hipcc() is None, reason="hipcc not available")
def test_ring_waits(tmp_path):
    out = tmp_path / "moe.s"
    cmd = [_hipcc(), "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", f"-I{os.path.join(ROOT, 'include')}", "-S", "--cuda-device-only", SRC, "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    waits, name, loads = {}, None, False
    for line in out.read_text().splitlines():
        m = re.match(r"(_Z\S*moe_(?:up|down)_kernel\S*):", line)
        if m:
            name, loads = m.group(1), False
            waits[name] = []
        elif ("s_barrier" in line or "s_endpgm" in line) and loads:
            name, loads = None, False
        elif name and "global_load_lds" in line:
            loads = True
        elif loads and (m := re.search(r"s_waitcnt .*vmcnt\((\d+)\)", line)):
            waits[name].append(int(m.group(1)))
    assert len(waits) >= 30
    for name, got in waits.items():
        rt, xn, slots = _cut(name)
        ring = [(slots - 2) * (rt + 1 + xn)]
        assert got == (ring if "moe_up" in name else ring + [0]), (name, got)
