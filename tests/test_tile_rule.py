"""Which kernel an int8 product takes and whether its launch stays below 2^32
threads, from the library's own rule."""
import pytest

from tile_rule import compile_rule


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    return compile_rule(str(tmp_path_factory.mktemp("rule")))


def test_launches_at_the_limit_of_threads(rule):
    # 16 channels and 512 threads a workgroup: up to 2^27 - 16 channels
    assert rule(1, (1 << 27) - 16, 16) == ("rows", (1 << 23) - 1, True)
    assert rule(1, (1 << 27) - 15, 16) == ("32x64", 1 << 21, True)
    assert rule(16, (1 << 27) + 5, 16).name == "32x64"
    # 512 threads a tile of 256 x 256: fewer than 2^23 tiles
    assert rule((1 << 31) - 1, 256, 64) == ("256x256", 1 << 23, False)
    assert rule((1 << 31) - 256, 256, 64) == ("256x256", (1 << 23) - 1, True)
    assert rule((1 << 30) - 1, 512, 64).fits is False
    # gated: 128 channels out of a tile's 256
    assert rule((1 << 30) - 1, 256, 64, gated=True).workgroups == 1 << 23
    # a tile more for every group
    assert rule(20 << 20, 2048, 4096, 1 << 20, grouped=True) == (
        "32x64", 32 * ((20 << 15) + (1 << 20)), False)


def test_choice_of_kernel(rule):
    assert rule(16, 4096, 7168).name == "rows"
    assert rule(16, 4096, 7168, 70000, grouped=True).name == "32x64"
    assert rule(17, 4096, 7168).name == "32x64"
    assert rule(8192, 4096, 7168).name == "256x256"
    assert rule(8192, 4096, 7168, wide=True).name == "64x64 wide"
    assert rule(32768, 2048, 4096, 72, gated=True, grouped=True).name == "128x256"
    assert rule(32768, 4096, 1024, 72, grouped=True).name == "256x256"
    assert rule(1500, 2111, 700).name == "128x128"
    assert rule(333, 1002, 1900).name == "32x64"
    assert rule(1000, 2048, 2048).name == "64x64"
