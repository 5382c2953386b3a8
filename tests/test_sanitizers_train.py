"""The host code of a training step's operators under AddressSanitizer + UndefinedBehaviorSanitizer
(tests/sanitize/driver_train.cpp, linked with the objects that tests/sanitize/build.py builds).  CPU only."""
import os
import subprocess

from quantized_routed_expert_moe_amd import build as B
from tests.sanitize import build as SB


def _build() -> str:
    SB.build()
    obj, exe = os.path.join(SB.OUT, "driver_train.o"), os.path.join(SB.OUT, "driver_train")
    cxx = os.path.join(SB.LLVM, "clang++")
    SB._run([cxx, "-std=c++17", *SB.SAN, "-fPIC", "-I" + os.path.join(SB.ROOT, "include"), "-c",
             os.path.join(SB.HERE, "driver_train.cpp"), "-o", obj])
    objs = [obj, *[os.path.join(SB.OUT, f) for f in ("abi.o", "abi_ops.o")],
            *[os.path.join(B.BUILD, os.path.splitext(s)[0] + ".o") for s in B.SOURCES if s not in ("abi.cpp", "abi_ops.cpp")],
            *[os.path.join(B.BUILD, f"ffn_prefill_{t}.o") for t in B.PREFILL_TYPES]]
    SB._run([cxx, *SB.SAN, *objs, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    return exe


def test_host_code_of_the_training_operators_is_clean():
    supp = os.path.join(SB.HERE, "lsan.supp")
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:halt_on_error=1",
               LSAN_OPTIONS=f"suppressions={supp}", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([_build()], capture_output=True, text=True, env=env, timeout=600)
    report = r.stdout + r.stderr
    assert r.returncode == 0, report[-4000:]
    assert "ERROR: AddressSanitizer" not in report and "runtime error" not in report, report[-4000:]
    assert "all passed" in r.stdout
