"""Build the sm_100a CUDA library in-tree (nvcc, no JIT), libfp8gemm.so, and the compiled part of the Python
binding (g++), _operators.so, next to this file."""
from __future__ import annotations

import importlib.util
import os
import pathlib
import subprocess
import sysconfig

HERE = pathlib.Path(__file__).resolve().parent
ROOT = HERE.parent
SO = HERE / "libfp8gemm.so"
SO_DEBUG = HERE / "libfp8gemm_debug.so"  # the same library with the device-side checks (-DFG_DEBUG)
BINDING = HERE / "_operators.so"  # marshalling of the operators (operators.py)
CSRC = HERE / "csrc"
COMMON = [CSRC / "fp8_cast_kernels.cuh", CSRC / "sm100_ptx.cuh", ROOT / "include" / "fp8gemm.h"]
# source -> what it includes
SOURCES = {
    CSRC / "fp8gemm_api.cu": COMMON + [CSRC / "fp8_gemm_kernels.cuh", CSRC / "fp8gemm_jit.h"],
    CSRC / "operators_api.cu": COMMON + [CSRC / "moe_route_kernels.cuh", CSRC / "moe_rows_kernels.cuh",
                                         CSRC / "lora_kernels.cuh", CSRC / "cluster_ptx.cuh"],
}

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


GEN = ROOT / "_build"
JIT_HEADERS = ["sm100_ptx.cuh", "fp8_gemm_kernels.cuh"]


def write_jit_sources() -> pathlib.Path:
    """Embed the kernel headers the library is built from, for its runtime-specialisation path
    (NVRTC compiles these exact sources): _build/fg_jit_sources.inc."""
    GEN.mkdir(exist_ok=True)
    parts = []
    for name in JIT_HEADERS:
        text = (HERE / "csrc" / name).read_text()
        assert ")FGJIT\"" not in text
        parts.append('R"FGJIT(' + text + ')FGJIT"')
    out = GEN / "fg_jit_sources.inc"
    body = ("// generated by moe_grouped_gemm_08_b200/build.py: the kernel headers, for runtime compilation\n"
            f"static const int kJitHeaderCount = {len(JIT_HEADERS)};\n"
            "static const char* const kJitHeaderNames[] = {" + ", ".join(f'"{n}"' for n in JIT_HEADERS) + "};\n"
            "static const char* const kJitHeaderSources[] = {\n" + ",\n".join(parts) + "};\n")
    if not out.exists() or out.read_text() != body:
        out.write_text(body)
    return out


def _newer(target: pathlib.Path, sources) -> bool:
    return target.exists() and target.stat().st_mtime >= max(p.stat().st_mtime for p in sources)


def _build_one(so: pathlib.Path, extra, force: bool, verbose: bool) -> pathlib.Path:
    """Compile the sources that changed to objects (side by side) and link them to `so`."""
    write_jit_sources()
    objects, running = [], []
    for src, includes in SOURCES.items():
        obj = GEN / f"{so.stem}.{src.stem}.o"
        objects.append(obj)
        if not force and _newer(obj, [src, *includes, pathlib.Path(__file__)]):
            continue
        tmp = obj.with_suffix(".o.tmp%d" % os.getpid())
        cmd = [nvcc(), *NVCC_FLAGS, *extra, "-I", str(ROOT / "include"), "-I", str(CSRC), "-I", str(GEN), "-c",
               str(src), "-o", str(tmp)]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        running.append((subprocess.Popen(cmd), cmd, tmp, obj))
    failed = [cmd for process, cmd, _, _ in running if process.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for _, _, tmp, obj in running:
        os.replace(tmp, obj)
    if running or not _newer(so, objects):
        tmp = so.with_suffix(".so.tmp%d" % os.getpid())
        subprocess.check_call([nvcc(), *NVCC_FLAGS, "-shared", "-ldl", *(str(o) for o in objects), "-o", str(tmp)])
        os.replace(tmp, so)
    return so


def torch_version() -> str:
    import torch
    return str(torch.__version__)


def binding_target() -> str:
    """What the binding is compiled against: torch's version and place, Python's ABI."""
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    return f"torch {torch_version()} at {torch}, {sysconfig.get_config_var('SOABI')}"


def build_binding(force: bool = False) -> pathlib.Path:
    """Compile the marshalling of the operators against the installed torch, linked to libfp8gemm.so beside it.  Built
    again when its sources are newer, and when torch or Python is another one than it was built for."""
    src = CSRC / "operators_binding.cpp"
    built_for, now = GEN / "operators_binding.built_for", binding_target()
    if (not force and _newer(BINDING, [src, ROOT / "include" / "fp8gemm.h", pathlib.Path(__file__)])
            and built_for.exists() and built_for.read_text() == now):
        return BINDING
    torch = pathlib.Path(importlib.util.find_spec("torch").submodule_search_locations[0])
    cuda = pathlib.Path(nvcc()).parent.parent if os.path.isabs(nvcc()) else pathlib.Path("/usr/local/cuda")
    includes = [ROOT / "include", sysconfig.get_paths()["include"], torch / "include", cuda / "include"]
    tmp = BINDING.with_suffix(".so.tmp%d" % os.getpid())
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f'-DFG_TORCH_VERSION="{torch_version()}"',
                           *(f"-I{i}" for i in includes), str(src), "-o",
                           str(tmp), f"-L{HERE}", "-l:libfp8gemm.so", "-Wl,-rpath,$ORIGIN", f"-L{torch / 'lib'}",
                           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
    os.replace(tmp, BINDING)
    GEN.mkdir(exist_ok=True)
    built_for.write_text(now)
    return BINDING


def build(force: bool = False, verbose: bool = False, debug: bool = True) -> pathlib.Path:
    """Compile the library (and, with debug=True, its debug build) if any source is newer than
    the built .so."""
    if debug:
        _build_one(SO_DEBUG, ["-DFG_DEBUG"], force, False)
    so = _build_one(SO, [], force, verbose)
    build_binding(force)
    return so


if __name__ == "__main__":
    print(build(force=True, verbose=True))
