"""The tiles of the 8-bit product without a GPU (tests/sanitize/q8_loads_driver.cpp):
where their loads go, under the address and undefined-behaviour sanitizers, and which
product takes which."""
import os
import shutil
import subprocess

import pytest

from q8_tile_cases import CASES

HERE = os.path.dirname(os.path.abspath(__file__))
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("q8") / "driver")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-g", "-Wall", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=undefined", os.path.join(HERE, "sanitize", "q8_loads_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="verify_asan_link_order=0")

    def run(*args):
        r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, env=env, timeout=300)
        assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
        return r.stdout.split("\n")[:-1]

    return run


def test_loads_stay_in_their_buffers(driver):
    """The scalar offset alone lies in the buffer for every load of every tile, and each lane reads its own element."""
    assert driver()[-1] == "ok"


def test_cases_reach_every_tile(driver):
    """The products of test_gpu_q8_tiles.py go to the tiles they are meant for, with fewer steps than are under way, as
    many, one more and more than twice as many: a new choice of tiles that loses one shows here."""
    chosen = [tuple(map(int, line.split())) for line in driver(*(v for c in CASES for v in c[1:]))]
    seen = set()
    for (tile, T, rows, cols), (got, ahead) in zip(CASES, chosen):
        assert got == tile, (T, rows, cols)
        steps = -(-cols // 128)
        seen.add((tile, "fewer" if steps < ahead else "as many" if steps == ahead else "one more" if steps == ahead + 1
                  else "more"))
        assert steps <= ahead + 1 or steps > 2 * ahead
    assert seen == {(t, n) for t in range(7) for n in ("fewer", "as many", "one more", "more")}
