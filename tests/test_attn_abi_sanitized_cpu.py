"""The host code of include/awq_attn.h's entry points under AddressSanitizer and UndefinedBehaviorSanitizer, as
test_abi_sanitized_cpu.py runs that of awq.h: the argument checks of test_attn_abi_cpu.py against the library built with both
on its host code, in a child process."""
import glob
import os
import subprocess
import sys
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.timeout(600)
def test_attn_host_code_is_clean_under_asan_and_ubsan():
    hits = sorted(glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"))
    if not hits or not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("no hipcc or clang sanitizer runtime")
    from post_quantization_mean_amd import build as bld

    lib = bld.build(sanitize=True)
    with tempfile.TemporaryDirectory() as logs:
        env = dict(os.environ)
        env["LD_PRELOAD"] = hits[-1] + (":" + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
        env["ASAN_OPTIONS"] = f"detect_leaks=0:log_path={logs}/asan"
        env["UBSAN_OPTIONS"] = f"print_stacktrace=1:halt_on_error=1:log_path={logs}/ubsan"
        code = ("import sys; sys.path.insert(0, %r)\n"
                "from post_quantization_mean_amd import binding as b\n"
                "b.load_library(%r)\n"
                "import pytest\n"
                "sys.exit(pytest.main(['-q', '-p', 'no:cacheprovider', '-m', 'not gpu', 'tests/test_attn_abi_cpu.py']))\n"
                ) % (ROOT, lib)
        r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True, text=True, timeout=500)
        logged = "".join(open(f, encoding="utf-8", errors="replace").read() for f in sorted(glob.glob(os.path.join(logs, "*"))))
        errors = "ERROR: AddressSanitizer" in logged or "runtime error:" in logged
        assert r.returncode == 0 and not errors, r.stdout[-3000:] + r.stderr[-3000:] + logged[:6000]
        assert "passed" in r.stdout
