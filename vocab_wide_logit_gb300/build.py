"""Build libdsample.so in-tree for sm_103a with nvcc (no CMake), and ds_calls.so, its short way from torch tensors.

The Gumbel bound table is generated first, then each translation unit is
compiled in parallel and linked into vocab_wide_logit_gb300/_build/libdsample.so,
which needs nvcc alone. Where torch is installed, ds_calls.so is built beside it.
"""
import concurrent.futures
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "_build")
LIB = os.path.join(OUT, "libdsample.so")
CALLS = os.path.join(OUT, "ds_calls.so")
INCLUDE = os.path.join(ROOT, "include")
SOURCES = ["ds_api.cu", "k_greedy.cu", "k_sample_warp.cu", "k_sample_cluster.cu", "k_sample_stream.cu",
           "k_merge.cu", "k_reveal.cu", "k_log_softmax.cu", "k_sample_filtered.cu", "k_quantize.cu",
           "k_linear_i8.cu", "k_score.cu", "k_score_grad.cu", "k_adapters.cu"]
HEADERS = ["ds_device.cuh", "ds_sample_common.cuh", "ds_warp_common.cuh", "ds_launch.h", "ds_index.h", "gen_gumbel_bounds.py"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def torch_identity():
    """What ds_calls.so depends on of the installed torch: its version file (None without torch)."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    with open(os.path.join(spec.submodule_search_locations[0], "version.py")) as f:
        return f.read()


def _calls_torch():
    """The torch_identity() that ds_calls.so was built with, None when that is not known."""
    try:
        with open(os.path.splitext(CALLS)[0] + ".torch") as f:
            return f.read()
    except OSError:
        return None


def _calls_command(src, out):
    """g++ for the CPython module, against the headers and libraries of the installed torch and CUDA runtime; None
    without torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    torch = spec.submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    inc = [INCLUDE, os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return (["g++", "-std=c++17", "-O2", "-fPIC", "-shared"] + ["-I" + i for i in inc] + [src, "-o", out,
            "-L" + os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    os.makedirs(OUT, exist_ok=True)
    table = os.path.join(OUT, "gumbel_bounds.inc")
    gen = os.path.join(CSRC, "gen_gumbel_bounds.py")
    if force or _stale(table, [gen]):
        subprocess.run([sys.executable, gen, table], check=True)
    common = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "dsample.h"), table,
                                                        os.path.abspath(__file__)]
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                    "-I", OUT, "--expt-relaxed-constexpr"]
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OUT, src.replace(".cu", ".o"))
        if force or ptxas_verbose or _stale(o, [s] + common):
            jobs.append([nvcc()] + flags + ["-c", s, "-o", o])
    src = os.path.join(CSRC, "py_calls.cpp")
    tmp_calls = CALLS + ".tmp%d" % os.getpid()
    calls, identity = None, torch_identity()
    deps = [src, os.path.join(INCLUDE, "dsample.h"), os.path.abspath(__file__)]
    if force or _stale(CALLS, deps) or _calls_torch() != identity:
        calls = _calls_command(src, tmp_calls)
        if calls is None:
            sys.stderr.write("torch is not installed: ds_calls.so (calls on torch tensors) is not built\n")
    failed = []
    commands = jobs + ([calls] if calls else [])
    if commands:
        with concurrent.futures.ThreadPoolExecutor(max_workers=len(commands)) as ex:
            results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), commands))
        for cmd, r in zip(commands, results):
            if verbose or ptxas_verbose or r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                failed.append(cmd)
    objs = [os.path.join(OUT, s.replace(".cu", ".o")) for s in SOURCES]
    if not any(cmd in failed for cmd in jobs) and (force or jobs or _stale(LIB, objs)):
        tmp = LIB + ".tmp%d" % os.getpid()
        subprocess.run([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"], check=True)
        os.replace(tmp, LIB)
    if calls and calls not in failed:
        os.replace(tmp_calls, CALLS)
        with open(os.path.splitext(CALLS)[0] + ".torch", "w") as f:
            f.write(identity)
    if failed:
        raise RuntimeError("compiler failed: " + "; ".join(" ".join(cmd) for cmd in failed))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="--ptxas" in sys.argv))
