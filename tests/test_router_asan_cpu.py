"""The host layer of the router's training operators and of the gradient norm (argument checks, overlap
checks, the plan's image) built with AddressSanitizer on its host code and driven by the CPU tests,
without a GPU."""
import glob
import os
import subprocess
import sys

import pytest

from test_host_asan_cpu import BUILD, PKG, ROOT, _asan_runtime, _hipcc

HOST = ("moe_api.hip", "router_api.hip")


def test_router_host_layer_under_address_sanitizer(tmp_path):
    hipcc, rt = _hipcc(), _asan_runtime()
    others = [o for o in glob.glob(os.path.join(BUILD, "*.hip.o")) if os.path.basename(o)[:-2] not in HOST]
    if not hipcc or not rt or not others:
        pytest.skip("needs hipcc, the clang sanitizer runtime and a previous build of the library")
    objs, lib = [], str(tmp_path / "libmoe_asan.so")
    inc = [f"-I{os.path.join(ROOT, 'include')}", f"-I{os.path.join(PKG, 'csrc')}"]
    cmds = []
    for src in HOST:
        objs.append(str(tmp_path / (src + ".o")))
        cmds.append([hipcc, "-O1", "-g", "-std=c++17", "--offload-arch=gfx950", "-fPIC", "-Xarch_host", "-fsanitize=address",
                     "-Xarch_host", "-fno-omit-frame-pointer", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *inc,
                     "-c", os.path.join(PKG, "csrc", src), "-o", objs[-1]])
    cmds.append([hipcc, "--offload-arch=gfx950", "-shared", "-fPIC", "-Xarch_host", "-fsanitize=address", "-shared-libsan",
                 "-o", lib, *objs, *others])
    for cmd in cmds:
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
    (tmp_path / "asan_library.py").write_text("import sparse_moe_layer_bailingmoev3_amd as m\n"
                                              f"m.lib_path = lambda: {lib!r}\n")
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:alloc_dealloc_mismatch=0:halt_on_error=1",
               PYTHONPATH=os.pathsep.join([str(tmp_path), ROOT, os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "asan_library", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_router_train_cpu.py")],
                       capture_output=True, text=True, env=env, cwd=ROOT, timeout=600)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert " passed" in out and "skipped" not in out.splitlines()[-1], out[-1000:]
