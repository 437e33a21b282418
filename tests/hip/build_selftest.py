"""Build the test-only libraries next to this file (hipcc for gfx950, same flags
as the product library): libnvfp4g_selftest.so, the GPU self-test, and
libi8_choice.so, the host's choice of tiles."""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(os.path.dirname(HERE))
sys.path.insert(0, ROOT)

from nvfp4_block_scaled_group_amd import build as B  # noqa: E402

LIB = os.path.join(HERE, "libnvfp4g_selftest.so")
CHOICE_LIB = os.path.join(HERE, "libi8_choice.so")


def _library(src: str, lib: str, verbose: bool) -> str:
    os.makedirs(B.BUILD_DIR, exist_ok=True)
    obj = os.path.join(B.BUILD_DIR, src + ".o")
    cmd = ["hipcc", *B.HIPCC_FLAGS, "-c", os.path.join(HERE, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    tmp = lib + ".tmp"
    subprocess.check_call(["g++", "-shared", "-o", tmp, obj, f"-L{B._hip_runtime_dir()}", "-lamdhip64",
                           f"-Wl,-rpath,{os.path.join(B.ROCM, 'lib')}", "-Wl,--no-undefined"])
    os.replace(tmp, lib)
    return lib


def build_choice(verbose: bool = False) -> str:
    return _library("i8_choice.hip", CHOICE_LIB, verbose)


def build(verbose: bool = False) -> str:
    build_choice(verbose)
    return _library("nvfp4_selftest.hip", LIB, verbose)


if __name__ == "__main__":
    print(build(verbose=True))
