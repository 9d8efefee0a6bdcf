"""Build libkda.so (the C ABI of include/kda.h) for gfx950 with hipcc, in-tree."""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libkda.so")
SOURCES = ["kda_api.hip", "kda_chunk.hip", "kda_chunk_logits.hip", "kda_chunk_logits_norm.hip", "kda_chunk_chain.hip", "kda_recurrent.hip", "kda_step.hip", "kda_gate.hip", "kda_util.hip", "kda_bwd.hip", "kda_noalloc.hip",
           "kda_gdr_api.hip", "kda_gdr_fwd.hip", "kda_gdr_bwd.hip", "kda_gdr_step.hip", "kda_draft_verify.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
         # no packed-fp32 instructions in device code
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include")]
# per-source extra flags: the DMA-fed chain kernel keeps its matrix-core accumulators in
# ordinary vector registers (the float32 state is rescaled by vector instructions every
# chunk; accumulation registers would need a move each way)
EXTRA = {"kda_chunk_chain.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
         "kda_gdr_fwd.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"], "kda_gdr_bwd.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}


def build(verbose: bool = False) -> str:
    obj_dir = os.path.join(HERE, "_build")
    os.makedirs(obj_dir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(obj_dir, src.replace(".hip", ".o"))
        cmd = [HIPCC, *FLAGS, *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("hipcc failed for %s:\n%s" % (src, r.stderr[-4000:]))
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s" % r.stderr[-4000:])
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
