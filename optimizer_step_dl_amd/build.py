"""Build libradamw.so (gfx950) in-tree with hipcc.

    python -m optimizer_step_dl_amd.build [-DNAME=VALUE ...] [--out PATH]

The HIP sources are compiled for gfx950 only.  Packed-FP32 instruction
selection is disabled (``-packed-fp32-ops``): the update is scalar FP32 per
element by design and the packed forms are not wanted here.
"""
from __future__ import annotations

import argparse
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(HERE, "libradamw.so")
SOURCES = ["radamw_balance.hip", "radamw_balance_sigmoid.hip",  # the longest first
           "radamw_residual_grad_f32_bf16.hip", "radamw_residual_grad_f32_f16.hip", "radamw_residual_grad.hip",
           "radamw_residual_grad_bf16.hip", "radamw_residual_grad_f16.hip", "radamw_residual.hip",
           "radamw_api.cpp", "radamw_update.hip", "radamw_stats.hip", "radamw_staged.hip", "radamw_probe.hip",
           "radamw_vocab_api.cpp", "radamw_embedding.hip", "radamw_loss.hip", "radamw_block_api.cpp", "radamw_dropout.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Wall", "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _run(cmd: list[str], quiet: bool) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed ({res.returncode}): {' '.join(cmd)}")
    if not quiet:
        sys.stderr.write(res.stderr)


def build(defines: list[str] | None = None, out: str | None = None, quiet: bool = True) -> str:
    """Compile the sources side by side, link them, and put the library in
    place when it is whole."""
    out = out or LIB_PATH
    common = [f"-I{INCLUDE}", f"-I{CSRC}", *[f"-D{d}" for d in (defines or [])]]
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, s + ".o") for s in SOURCES]
        with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            jobs = [pool.submit(_run, [HIPCC, *FLAGS, *common, "-x", "hip", "-c", os.path.join(CSRC, s), "-o", o], quiet)
                    for s, o in zip(SOURCES, objects)]
            for j in jobs:
                j.result()
        _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objects, "-o", out + ".tmp"], quiet)
    os.replace(out + ".tmp", out)
    return out


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("-D", dest="defines", action="append", default=[])
    ap.add_argument("--out", default=None)
    args = ap.parse_args(argv)
    print(build(args.defines, args.out, quiet=False))


if __name__ == "__main__":
    main()
