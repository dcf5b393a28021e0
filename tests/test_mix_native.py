"""The channel-mixing entry points' host logic (validation, choice of shapes,
workspace sizing, pointer checks) under AddressSanitizer and
UndefinedBehaviorSanitizer, driven by ``native/mix_sanitize.c``; no kernel is
launched."""
import os
import subprocess

import pytest


def test_mix_host_logic_under_asan_and_ubsan():
    native = pytest.importorskip("test_native_host")
    native._build_sanitized()        # the library's objects
    out = os.path.join(native.BUILD, "asan")
    objs = [os.path.join(out, os.path.basename(s) + ".o") for s in native._sources()]
    cc, drv, exe = native.hipcc(), os.path.join(out, "mix_sanitize.o"), os.path.join(out, "mix_sanitize")
    for cmd in ([cc, "-x", "c++", "-O1", "-std=c++17"] + native.SAN[:4] +
                ["-c", os.path.join(native.NATIVE, "mix_sanitize.c"), "-o", drv],
                [cc, "--offload-arch=gfx950"] + native.SAN + objs + [drv, "-o", exe]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and r.stdout.startswith("ok "), (r.stdout + r.stderr)[-6000:]
    assert int(r.stdout.split()[1]) > 30000
