"""How the few-token expert layer cuts a call, compiled for the host: over all
numbers of tokens and choices, and experts, widths and formats from end to end of
their ranges, the workgroups fit in LDS and the lists and parts in the workspace.
(A call that did not fit would be refused by the launch, not by a rule.)"""
import os
import shutil
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
NAMES = ("fmt hidden tokens top_k experts segment dmas most_segments down_tiles splits up_lds down_lds segment_room "
         "part_room").split()


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    cxx = shutil.which("hipcc")
    if cxx is None:
        pytest.skip("hipcc not available")
    d = tmp_path_factory.mktemp("moe")
    exe, out = str(d / "moe_plan_dump"), str(d / "dump.bin")
    subprocess.run([cxx, "-O2", "-std=c++17", "-o", exe, os.path.join(HERE, "host", "moe_plan_dump.cpp")], check=True,
                   capture_output=True)
    subprocess.run([exe, out], check=True)
    return dict(zip(NAMES, np.fromfile(out, dtype=np.int32).reshape(-1, len(NAMES)).T.astype(np.int64)))


def test_workgroups_fit_in_lds(plans):
    assert plans["up_lds"].max() <= 160 * 1024 and plans["down_lds"].max() <= 160 * 1024


def test_lists_and_parts_fit_in_the_workspace(plans):
    p = plans
    rows = p["tokens"] * p["top_k"]
    # any routing: full segments, and one that is not full for each chosen expert
    assert (p["most_segments"] >= rows // p["segment"] + np.minimum(rows, p["experts"])).all()
    assert (p["most_segments"] <= p["segment_room"]).all()
    split = p["splits"] > 1
    assert (p["splits"] * p["tokens"] * p["hidden"] <= p["part_room"])[split].all() and (p["splits"] >= 1).all()


def test_segments_are_whole_loads_of_one_mfma(plans):
    p = plans
    each = np.where(p["fmt"] == 0, 4, 8)                   # tokens that a load brings a piece of
    assert (p["segment"] == p["dmas"] * each).all() and (p["segment"] <= 16).all() and (p["dmas"] >= 1).all()
    assert set(np.unique(p["down_tiles"])) == {1, 4} and not ((p["down_tiles"] == 1) & (p["splits"] > 1)).any()
