"""Places in the exchange buffer of the norms' kernels, enumerated on the host: the heads of a warp store all of their words
between two barriers, so that no two may share a place."""
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("norm_exchange") / "check")
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "dit_modulate_absmax_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "helpers", "norm_exchange_check.cpp"), "-o", exe], check=True)
    words, *rows = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    return int(words), np.array([r.split() for r in rows], dtype=np.int64)


@pytest.mark.parametrize("dim", range(8, 257, 8))
def test_every_word_has_a_place_of_its_own(places, dim):
    words, all_ = places
    mine = all_[all_[:, 1] == dim]
    lanes = 4 if dim <= 64 else 8 if dim <= 128 else 16
    assert (mine[:, 0] == lanes).all() and len(mine) == 32 // lanes * dim // 2
    assert len(np.unique(mine[:, 4])) == len(mine)
    assert mine[:, 4].min() >= 0 and mine[:, 4].max() < words


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_the_lanes_words_fall_into_different_banks(places, dim):
    """A warp's stores, of whole heads: word i of the lanes' first chunks of four, then of their second."""
    _, all_ = places
    mine = all_[all_[:, 1] == dim]
    for chunk in (0, 1):
        for i in range(4):
            words = mine[(mine[:, 3] >= chunk * dim // 4) & (mine[:, 3] < (chunk + 1) * dim // 4) & (mine[:, 3] % 4 == i)]
            assert len(words) == 32 and len(np.unique(words[:, 4] % 32)) == 32
