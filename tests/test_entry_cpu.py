"""The C entry points of cross-attention and of the heads' norm and rotation, compiled
for the host against stand-ins for the CUDA runtime and the launches
(tests/cuda/entry_fakes.cpp): what they do behind their first CUDA call."""
import ctypes
import os
import random
import re
import shutil
import subprocess
import sys

import pytest

from exact_attention_68_gb300 import binding, cross, rope
from exact_attention_68_gb300.build import CSRC, ROOT, _nvcc

CUDA_ERROR = 100  # cudaErrorNoDevice


@pytest.fixture(scope="module")
def entry(tmp_path_factory):
    """The path of the library of entry points and stand-ins."""
    to = str(tmp_path_factory.mktemp("entry") / "libentry.so")
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    r = subprocess.run([cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                        "-I", cuda, "-x", "c++", os.path.join(CSRC, "cross_api.cu"), os.path.join(CSRC, "rope_api.cu"),
                        os.path.join(ROOT, "tests", "cuda", "entry_fakes.cpp"), "-o", to], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return to


def load(path):
    lib = rope.declare(cross.declare(ctypes.CDLL(path)))
    lib.fake_device(152, 0)
    return lib


A, T = 0x700000000000, 1 << 36  # device addresses that nobody reads


def cross_fwd(lib, sizes, ws=A + 20 * T, space=1 << 34):
    return lib.attn_cross_fwd(cross._pack_sizes(*sizes), A, A + T, A + 2 * T, None, A + 3 * T, A + 4 * T, 0.125, 0, ws, space,
                              0, None)


def cross_bwd(lib, sizes, ws=A + 20 * T, space=1 << 34):
    return lib.attn_cross_bwd(cross._pack_sizes(*sizes), *(A + i * T for i in range(3)), None, *(A + i * T for i in range(3, 10)),
                              0.125, 0, ws, space, 0, None)


def rope_call(lib, bwd, ws=A + 20 * T, space=1 << 34):
    B, S, H, D = 2, 16, 4, 64
    part = rope._pack_part(A, S * H * D, H * D, D, H, A + T, 0, 0, A + 2 * T, A + 3 * T, S * H * D, H * D, D, A + 4 * T)
    if bwd:
        return lib.attn_rope_bwd(part, 1, None, None, B, S, D, 1e-6, 0, ws, space, None)
    return lib.attn_rope_fwd(part, 1, None, None, B, S, D, 1e-6, 0, None)


SIZES = {"few": (2, 4, 2, 1, 900, 64), "tiles": (2, 4, 2, 300, 900, 128), "wide": (2, 4, 2, 300, 900, 256),
         "small": (2, 2, 2, 20, 40, 64)}
CALLS = {**{f"{n}_{name}": (lambda lib, f=f, s=s: f(lib, s)) for n, f in (("fwd", cross_fwd), ("bwd", cross_bwd))
            for name, s in SIZES.items()},
         "rope_fwd": lambda lib: rope_call(lib, False), "rope_bwd": lambda lib: rope_call(lib, True)}


def test_sound_calls_launch(entry):
    lib = load(entry)
    for name, call in CALLS.items():
        lib.fake_device(152, 0)
        assert call(lib) == binding.ATTN_OK and lib.fake_launches() > 0, name


def test_device_queries_that_fail_are_errors(entry):
    """Not divisions by the SMs that they did not tell.  In a process of its own, which such a division would end."""
    code = ("import test_entry_cpu as t, sys\n"
            "lib = t.load(sys.argv[1])\n"
            "for name, call in t.CALLS.items():\n"
            "    lib.fake_device(152, t.CUDA_ERROR)\n"
            "    print(name, call(lib), lib.fake_cuda_error(), lib.fake_launches(), flush=True)\n")
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    r = subprocess.run([sys.executable, "-c", code, entry], capture_output=True, text=True, env=env, cwd=ROOT)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr[-500:])
    assert r.stdout.split("\n")[:-1] == [f"{name} {binding.ATTN_ERR_CUDA} {CUDA_ERROR} 0" for name in CALLS]


def test_workspace_queries_without_a_device(entry):
    lib = load(entry)
    lib.fake_device(152, CUDA_ERROR)
    for s in SIZES.values():
        packed = cross._pack_sizes(*s)
        assert lib.attn_cross_fwd_workspace(packed) == 0 and lib.attn_cross_bwd_workspace(packed) == 0


def test_workspace_queries_tell_what_the_calls_need(entry):
    """Over random sizes: what the query says is enough, and a byte less is not."""
    lib, rng, needed = load(entry), random.Random(5), 0
    for _ in range(1500):
        G, Hkv, D = rng.choice([1, 1, 2, 8]), rng.choice([1, 2, 5, 16]), rng.randrange(8, 257, 8)
        sizes = (rng.choice([1, 1, 2, 9]), G * Hkv, Hkv, int(2 ** rng.uniform(0, 11)), int(2 ** rng.uniform(0, 14)), D)
        for call, query in ((cross_fwd, lib.attn_cross_fwd_workspace), (cross_bwd, lib.attn_cross_bwd_workspace)):
            need = query(cross._pack_sizes(*sizes))
            assert need >= 16
            assert call(lib, sizes, space=need) == binding.ATTN_OK, sizes
            if need > 16:
                needed += 1
                assert call(lib, sizes, space=need - 1) == binding.ATTN_ERR_INVALID_ARG, sizes
                assert call(lib, sizes, ws=A + 20 * T + 8, space=need) == binding.ATTN_ERR_MISALIGNED, sizes
    assert needed > 500


def test_cluster_barriers_take_diverged_warps():
    """They stand behind loops that a warp's threads leave one by one, where the aligned form is undefined."""
    found = 0
    for name in os.listdir(CSRC):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        found += text.count("barrier.cluster.arrive")
        assert not re.search(r"barrier\.cluster\.(arrive|wait)[.\w]*\.aligned", text), name
    assert found >= 2
