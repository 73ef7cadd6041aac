"""Build libkvc.so in-tree for sm_103a (nvcc, translation units compiled in parallel), and the Python binding's
native marshalling module (g++ against torch's headers)."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libkvc.so")
CALL_PATH = os.path.join(OUT_DIR, "_kvc_call.so")
CALL_STAMP = CALL_PATH + ".abi"   # what _kvc_call.so was built against, see call_abi
ROOT = os.path.dirname(HERE)

SOURCES = ["kvc_core.cu", "kvc_attn.cu", "kvc_decode_bf16.cu", "kvc_decode_fp8.cu", "kvc_decode_int4.cu",
           "kvc_decode_tc.cu", "kvc_decode_tc8.cu", "kvc_prefill_tc.cu", "kvc_noalloc.cu", "kvc_alloc.cu", "kvc_rope.cu",
           "kvc_mod.cu", "kvc_mod_bf16.cu", "kvc_mod_fp8.cu", "kvc_mod_int4.cu", "kvc_mod_tc.cu", "kvc_mod_tcq.cu",
           "kvc_plan.cu", "kvc_select.cu", "kvc_select_tc.cu", "kvc_sparse.cu", "kvc_sparse_q.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden", "--expt-relaxed-constexpr",
              "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def call_abi() -> str:
    """What the marshalling module depends on beside its sources: torch's C++ classes and the interpreter's objects."""
    import sysconfig
    import torch
    return f"torch {torch.__version__} {os.path.dirname(torch.__file__)} python {sysconfig.get_config_var('SOABI')}"


def call_current() -> bool:
    """Whether the marshalling module was built against the torch and Python that run now."""
    try:
        with open(CALL_STAMP) as f:
            return f.read() == call_abi()
    except OSError:
        return False


def call_stale() -> bool:
    """Whether the marshalling module is missing, older than its sources, or built against another torch or Python."""
    sources = [os.path.join(CSRC, "kvc_call.cpp"), os.path.join(ROOT, "include", "kvc.h")]
    return _stale(CALL_PATH, sources) or not call_current()


def _replace(path: str, make) -> None:
    """make(temporary path), then the file takes its place at once: a process that has the old one mapped keeps it."""
    tmp = f"{path}.tmp{os.getpid()}"
    try:
        make(tmp)
        os.replace(tmp, path)
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)


def call_commands(out: str = CALL_PATH) -> tuple[list[str], list[str]]:
    """Compile and link commands of the marshalling module, through out + ".o"."""
    import sysconfig
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    obj = out + ".o"
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + os.path.join(home, "include"),
                "-I" + os.path.join(home, "include", "torch", "csrc", "api", "include"),
                "-I" + os.path.join(cuda, "include"), "-I" + sysconfig.get_paths()["include"],
                "-c", os.path.join(CSRC, "kvc_call.cpp"), "-o", obj]
    link = ["g++", "-shared", "-o", out, obj, "-L" + OUT_DIR, "-l:libkvc.so", "-Wl,-rpath,$ORIGIN",
            "-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    return compile_, link


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(ROOT, "include", "kvc.h"))
    flags = NVCC_FLAGS + (extra_flags or [])
    procs, objs = [], []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [path] + headers):
            cmd = [nvcc()] + ARCH + flags + ["-c", path, "-o", obj]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    call = force or call_stale()
    call_tmp = f"{CALL_PATH}.tmp{os.getpid()}"
    if call:
        procs.append(("kvc_call.cpp", subprocess.Popen(call_commands(call_tmp)[0], stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if failed:
        if os.path.exists(call_tmp + ".o"):
            os.remove(call_tmp + ".o")
        raise RuntimeError("nvcc failed:\n" + "\n".join(f"--- {s}\n{o}" for s, o in failed))
    if force or procs or _stale(LIB_PATH, objs):
        _replace(LIB_PATH, lambda tmp: subprocess.check_call(
            [nvcc()] + ARCH + ["-shared", "-Xlinker", "-z,defs", "-o", tmp] + objs))
    if call:
        _replace(CALL_PATH, lambda tmp: subprocess.check_call(call_commands(tmp)[1]))   # the object made above
        os.remove(call_tmp + ".o")
        with open(CALL_STAMP, "w") as f:   # last: without it the module counts as stale
            f.write(call_abi())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
