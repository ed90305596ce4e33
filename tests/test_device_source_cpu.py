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


HELPER = re.compile(r"__forceinline__\s+[\w:<>\s*&]*?\b(\w+)\s*\(")


@pytest.mark.parametrize("name", list(SOURCES))
def test_every_device_helper_is_called(name):
    everything = "\n".join(SOURCES.values())
    for helper in set(HELPER.findall(SOURCES[name])):
        if helper[0].isupper():  # a constructor
            continue
        defined = HELPER.findall(everything).count(helper)
        assert len(re.findall(rf"\b{helper}\b", everything)) > defined, helper


def test_instruction_wrappers_have_one_form():
    """An overload that nothing calls hides behind its name."""
    helpers = HELPER.findall(SOURCES["expert_ptx.cuh"])
    assert len(helpers) > 30 and len(set(helpers)) == len(helpers)


def test_no_instruction_is_wrapped_for_a_pair_that_nobody_asks_for():
    """Wrappers with a form for one CTA and one for a pair are called with both."""
    everything = "\n".join(SOURCES.values())
    both = re.findall(r"template <int CG[^>]*>\s*__device__ __forceinline__ \w+ (\w+)\(",
                      SOURCES["expert_ptx.cuh"])
    assert len(both) >= 5
    for helper in both:
        forms = set(re.findall(rf"\b{helper}<(\w+)", everything))
        assert "CG" in forms or "2" in forms, helper
