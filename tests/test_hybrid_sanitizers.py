"""The C entry points of include/lfm2sc_hybrid.h under AddressSanitizer and UndefinedBehaviorSanitizer, host code only (CPU).

api_hybrid.cpp (argument checks, workspace sizes, dispatch), api.cpp and the host halves of the kernels' files (plans, grids)
are compiled with the host sanitizers and linked with the library's other objects into a temporary directory; the entry
points' tests, the binding's and the size limits' then run in a child process that loads the sanitizer runtime first.  Any
report ends it.
"""
import concurrent.futures as cf
import os
import subprocess
import sys

import pytest

from gated_short_causal_amd import build
from test_host_sanitizers import BUILD, CSRC, HIPCC, ROOT, _run, _runtime

CHECKED = ["api.cpp", "api_hybrid.cpp", "attn_fwd.hip", "attn_bwd.hip", "attn_cached.hip", "drafts.hip", "check.hip"]
TESTS = ["tests/test_hybrid_abi.py", "tests/test_hybrid_binding.py", "tests/test_hybrid_binding_rows.py", "tests/test_hybrid_limits.py"]


def test_hybrid_host_code_under_asan_ubsan(tmp_path):
    rt = _runtime()
    if rt is None or not os.path.exists(HIPCC):
        pytest.skip("clang sanitizer runtime or ROCm compilers not found")
    others = [os.path.join(BUILD, s + ".o") for s in build.SOURCES if s not in CHECKED]
    missing = [o for o in others if not os.path.exists(o)]
    if missing:
        pytest.skip(f"library objects not built yet ({missing}): run __graft_entry__.build() first")
    host = [x for flag in ("-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer")
            for x in ("-Xarch_host", flag)]

    def compile_one(src):
        obj = str(tmp_path / (src + ".o"))
        _run([HIPCC, *build.compile_flags(), "-O1", *host, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj])
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(CHECKED)) as ex:
        objs = list(ex.map(compile_one, CHECKED))
    lib = str(tmp_path / "liblfm2sc_san.so")
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", lib, *objs, *others])
    nm = _run(["nm", "-D", lib]).stdout
    assert "__asan_" in nm and "__ubsan_" in nm, "the host code was not instrumented"

    env = dict(os.environ)
    env["LD_PRELOAD"] = rt + (" " + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
    env["ASAN_OPTIONS"] = "detect_leaks=0:abort_on_error=1"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    env["LFM2SC_LIB"] = lib
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", *TESTS], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, f"sanitized run failed:\n{r.stdout[-4000:]}\n{r.stderr[-4000:]}"
    assert "passed" in r.stdout and "failed" not in r.stdout, r.stdout[-2000:]
