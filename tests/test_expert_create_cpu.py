"""moe_expert_create prepares the kernels that its handle can launch and no others: what
another type's kernels need must not decide whether a handle can be made. The CUDA runtime
calls are fakes that note the kernels (fake_cuda_runtime.c), in a process of their own."""
import json
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

KINDS = {"bf16": (0, 0), "bf16_train": (0, 1), "e4m3": (1, 0), "int8": (2, 0)}

CHILD = """
import ctypes, json, sys
sys.path.insert(0, {root!r})
from combine_top_histogram_gb300 import binding as B
fake, lib = ctypes.CDLL({fake!r}), B.load_library()
def create(dtype, train):
    cfg, h = B.make_expert_config(4, 256, 128, 64, dtype, train), ctypes.c_void_p()
    rc = lib.moe_expert_create(ctypes.byref(cfg), ctypes.c_void_p(256), 1 << 30, ctypes.byref(h))
    buf = (ctypes.c_void_p * 1024)()
    return rc, set(buf[:fake.fake_opted(buf)])
kinds = {kinds!r}
sets = {{name: create(*v) for name, v in kinds.items()}}
refused = {{}}
for name in kinds:
    for other in kinds:
        for f in sets[other][1] - sets[name][1]:
            fake.fake_refuse(ctypes.c_void_p(f))
            refused.setdefault(name, set()).add(create(*kinds[name])[0])
    own = next(iter(sets[name][1]))
    fake.fake_refuse(ctypes.c_void_p(own))
    refused[name + " own"] = {{create(*kinds[name])[0]}}
    fake.fake_refuse(None)
print(json.dumps({{"rc": {{n: v[0] for n, v in sets.items()}},
                   "sets": {{n: sorted(v[1]) for n, v in sets.items()}},
                   "refused": {{n: sorted(v) for n, v in refused.items()}}}}))
"""


@pytest.fixture(scope="module")
def created(cuda_lib, tmp_path_factory):
    from importlib import import_module
    build = import_module("combine_top_histogram_gb300.build")
    include = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    fake = str(tmp_path_factory.mktemp("fake") / "libfakecuda.so")
    subprocess.check_call(["gcc", "-O1", "-shared", "-fPIC", "-I", include, "-o", fake,
                           os.path.join(HERE, "fake_cuda_runtime.c")])
    code = CHILD.format(root=build.ROOT, fake=fake, kinds=KINDS)
    out = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, LD_PRELOAD=fake),
                         stdout=subprocess.PIPE, check=True, timeout=120).stdout
    return json.loads(out.decode().splitlines()[-1])


def test_every_kind_of_handle_is_made(created):
    assert set(created["rc"].values()) == {0}
    assert all(created["sets"][kind] for kind in KINDS)


@pytest.mark.parametrize("a, b", [("bf16", "e4m3"), ("bf16", "int8"), ("e4m3", "int8"),
                                  ("bf16_train", "e4m3"), ("bf16_train", "int8")])
def test_types_share_no_kernel(created, a, b):
    assert not set(created["sets"][a]) & set(created["sets"][b])


def test_backward_kernels_belong_to_training(created):
    assert set(created["sets"]["bf16"]) < set(created["sets"]["bf16_train"])


@pytest.mark.parametrize("kind", list(KINDS))
def test_another_types_kernel_refuses_no_handle(created, kind):
    assert created["refused"][kind] == [0]
    assert created["refused"][kind + " own"] == [-4]
