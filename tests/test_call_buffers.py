"""Which buffers of a call may share memory: the library's check, built for the host
with g++, against the rule by bytes (CPU only)."""
import itertools
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def may_run(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("buffers") / "buffers_host")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Werror", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", os.path.join(ROOT, "tests", "host", "buffers_host.cpp"), "-o", exe], check=True)

    def run(*buffers):
        args = [":".join(map(str, b)) for b in buffers]
        return subprocess.run([exe, *args], check=True, capture_output=True, text=True).stdout.strip() == "1"
    return run


IN, OUT, NONE = 0, 1, -1


def test_an_output_may_be_its_partner_and_nothing_else(may_run):
    """Combine's X, R and Y, and the weight gradient's D, A, base and dB: Y may be R and
    dB its base, but not where X (D, A) has that address too."""
    x, r, other = 4096, 8192, 16384
    assert may_run((x, 512, IN, NONE), (r, 512, IN, NONE), (r, 512, OUT, 1))
    assert may_run((x, 512, IN, NONE), (x, 512, IN, NONE), (r, 512, OUT, 1))
    assert not may_run((x, 512, IN, NONE), (x, 512, IN, NONE), (x, 512, OUT, 1))
    assert not may_run((x, 512, IN, NONE), (r, 512, IN, NONE), (x, 512, OUT, 1))
    assert not may_run((x, 512, IN, NONE), (0, 0, IN, NONE), (x, 512, OUT, 1))  # an empty partner
    for taken in (0, 1):
        at = [other, other + 4096, x, x]
        assert may_run(*((p, 512, int(i == 3), 2 if i == 3 else NONE) for i, p in enumerate(at)))
        at[taken] = x
        assert not may_run(*((p, 512, int(i == 3), 2 if i == 3 else NONE) for i, p in enumerate(at)))


def test_all_places_of_three_buffers(may_run):
    """Every placing of an input, a partner and an output on a few bytes."""
    for a, b, c, n in itertools.product(range(0, 4), range(0, 4), range(0, 4), (1, 2)):
        def meet(p, pn, q, qn):
            return p < q + qn and q < p + pn
        want = not meet(c, n, a, 2) and (c == b or not meet(c, n, b, n))
        assert may_run((64 + a, 2, IN, NONE), (64 + b, n, IN, NONE), (64 + c, n, OUT, 1)) == want, (a, b, c, n)
