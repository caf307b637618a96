"""Build libufp4.so (all HIP sources, gfx950 only) in the package directory."""
from __future__ import annotations

import os
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

_HERE = os.path.dirname(os.path.abspath(__file__))
SOURCES = [os.path.join(_HERE, "csrc", f)
           for f in ("ufp4_quant.hip", "ufp4_misc.hip", "ufp4_gemm.hip", "ufp4_host.hip", "ufp4_api.hip",
                     "ufp4_expert.hip", "ufp4_ckpt.hip", "ufp4_grouped.hip", "ufp4_moe_api.hip")]
OUT = os.path.join(_HERE, "libufp4.so")

# -ffp-contract=off: no implicit fused multiply-add (every rounding step is
# the one written).  The packed-fp32 feature is disabled: the kernels never
# use packed binary32 instructions.
HIPCC_FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
               "-ffp-contract=off", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-Wall"]


def hipcc() -> str:
    return shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


def _run(cmd: list) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    msg = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                    if "packed-fp32-ops' is not a recognized feature" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed:\n{msg}")
    return msg


def build(verbose: bool = False) -> str:
    """Compiles every source to an object, side by side, and links them."""
    with tempfile.TemporaryDirectory(prefix="ufp4_build_") as tmp:
        objects = [os.path.join(tmp, os.path.basename(f) + ".o") for f in SOURCES]
        cmds = [[hipcc()] + [f for f in HIPCC_FLAGS if f != "-shared"] + ["-c", "-o", o, f]
                for f, o in zip(SOURCES, objects)]
        cmds.append([hipcc()] + HIPCC_FLAGS + ["-o", OUT + ".tmp"] + objects)
        if verbose:
            print("\n".join(" ".join(c) for c in cmds), flush=True)
        with ThreadPoolExecutor(max_workers=4) as pool:
            msgs = list(pool.map(_run, cmds[:-1]))
        msgs.append(_run(cmds[-1]))
    for msg in msgs:
        if verbose and msg.strip():
            print(msg)
    os.replace(OUT + ".tmp", OUT)
    return OUT


if __name__ == "__main__":
    print(build(verbose=True))
