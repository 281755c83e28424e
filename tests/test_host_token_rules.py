"""The rules of the token and int8 operators, compiled for the host."""
import os
import shutil
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    """rules(mode, columns, *args): the rows that a mode writes."""
    cxx = shutil.which("hipcc")
    if cxx is None:
        pytest.skip("hipcc not available")
    d = tmp_path_factory.mktemp("token")
    exe, out = str(d / "token_rules_dump"), str(d / "dump.bin")
    subprocess.run([cxx, "-O2", "-std=c++17", "-o", exe, os.path.join(HERE, "host", "token_rules_dump.cpp")], check=True,
                   capture_output=True)

    def run(mode, columns, *args):
        subprocess.run([exe, mode, out, *map(str, args)], check=True)
        return np.fromfile(out, dtype=np.int32).reshape(-1, columns)
    return run


def test_a_columns_gradient_is_stored_by_one_lane(rules):
    """What a lane of combine's gradient stores where that goes over y, elements start +
    skip up to start + n, is no other lane's, and all together are the row. (One that
    stored its neighbour's elements would do so before another wave has read them.)
    What it loads lies inside the row."""
    n, cols, col, start, skip = rules("chunks", 5).T.astype(np.int64)
    assert (start >= 0).all() and (start + n <= cols).all() and (skip >= 0).all() and (skip < n).all()
    first = start + skip
    assert (first == col).all()
    last = np.minimum(col + n, cols)
    assert (start + n == last).all()
    # chunk after chunk of one row, each begins where the one before it ends
    same = cols[1:] == cols[:-1]
    assert (first[1:][same] == last[:-1][same]).all() and (last[:-1][~same] == cols[:-1][~same]).all()


def test_pieces_of_any_number_of_tokens(rules):
    """Tiles of an expert's tokens, up to the most rows that the product takes."""
    m, each, pieces = rules("pieces", 3, 0, 1, 15, 16, 17, 255, 256, 257, 10 ** 6, 2 ** 30, 2 ** 31 - 257, 2 ** 31 - 256,
                            2 ** 31 - 255, 2 ** 31 - 128, 2 ** 31 - 1).T.astype(np.int64)
    assert (pieces == -(-m // each)).all() and len(m) == 75


@pytest.mark.parametrize("cus", [256])
def test_every_form_of_the_int8_product_is_run(rules, cus):
    """The library's own rule takes every form for one of the shapes that the product
    is tested at on the GPU."""
    from . import test_gpu_int8 as gpu
    shapes = [m for m in gpu.test_product.pytestmark if m.name == "parametrize"][0].args[1]
    forms = [rules("form", 2, cus, N, K, *splits)[0] for splits, N, K in shapes]
    assert {f for f, _ in forms} == set(range(forms[0][1]))


def test_forms_of_few_tokens_fit_the_grid(rules):
    """Their pieces are the grid's second axis, 65535 at most."""
    heights = {2: 16, 4: 16, 3: 32, 5: 32, 7: 32, 6: 64, 8: 64}
    for each in (16, 32, 64):
        for m in (65535 * each, 65535 * each + 1):
            for splits in ([m], [1, 0, m - 1], [m // 3] * 3):
                for N, K in ((1, 16), (16, 131056), (64, 4096)):
                    form = int(rules("form", 2, 256, N, K, *splits)[0][0])
                    assert form < 2 or sum(-(-v // heights[form]) for v in splits) <= 65535, (splits, N, K, form)
