"""The experts' product refuses sizes that its kernels would count past an int: the
library's own limits, built for the host with g++ (CPU only)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST = 2 ** 31 - 1
# heights and widths of the kernels' tiles
HEIGHTS, WIDTHS = (16, 32, 64, 128, 256), (32, 64, 128, 256)


def counted(rows, n, experts):
    """What the kernels add up in ints stays in range: a size with a tile more, and an
    expert's tiles of every shape."""
    return all(rows + h <= MOST and n + w <= MOST and (rows // h + experts) * -(-n // w) <= MOST
               for h in HEIGHTS for w in WIDTHS)


@pytest.fixture(scope="module")
def taken(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("limits") / "limits_host")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Werror", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", os.path.join(ROOT, "tests", "host", "limits_host.cpp"), "-o", exe], check=True)

    def run(sizes):
        out = subprocess.run([exe, *(str(v) for s in sizes for v in s)], check=True, capture_output=True, text=True).stdout
        return [line == "1" for line in out.split()]
    return run


def test_what_is_taken_is_counted(taken):
    edges = [1, 15, 16, 4096, 2 ** 24, 2 ** 30] + [MOST - d for d in (512, 257, 256, 255, 127, 63, 31, 15, 0)]
    sizes = [(r, n, e) for r in edges for n in edges for e in (1, 2, 1024)]
    got = taken(sizes)
    assert any(got) and not all(got)
    for size, yes in zip(sizes, got):
        assert not yes or counted(*size), size


def test_limits(taken):
    """One row of the widest matrix is taken, a column more is not."""
    assert taken([(1, MOST - 256, 1), (1, MOST - 255, 1), (1, MOST, 1)]) == [True, False, False]
    assert taken([(MOST - 256, 16, 1), (MOST - 255, 16, 1)]) == [True, False]
    assert taken([(65536, 4096, 64), (13000, 130, 1000)]) == [True, True]
