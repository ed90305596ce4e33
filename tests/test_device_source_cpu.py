"""What the device sources must hold and no run on a GPU can show: behaviour that PTX leaves
undefined and a compiler may get right by chance (no GPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "combine_top_histogram_gb300", "csrc")


def code(name):
    """A source without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


SOURCES = {name: code(name) for name in sorted(os.listdir(CSRC))}


@pytest.mark.parametrize("name", list(SOURCES))
def test_lanes_converge_before_an_aligned_cluster_barrier(name):
    """barrier.cluster.arrive.aligned needs every lane of a warp at the same instruction, and
    the barrier follows stores and arrivals of single lanes: a __syncwarp stands right before it."""
    for part in re.split(r"barrier\.cluster\.arrive", SOURCES[name])[:-1]:
        last = [s.strip() for s in part.split(";") if s.strip()][-2]
        assert last.endswith("__syncwarp()"), last[-80:]
