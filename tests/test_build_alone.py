"""The library builds for a user of the C ABI or the FFN binding alone, who
needs neither torch nor Python's headers."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_build_without_torch():
    r = run("import sys; sys.modules['torch'] = None\n"
            "from moe_decode_layer_sm_b200 import build, lib\n"
            "assert not build.can_build_call() and build.build() == build.SO\n"
            "assert lib().mono_ffn_abi_version() > 0")
    assert r.returncode == 0, r.stderr


def test_build_without_headers(tmp_path):
    r = run("import sysconfig\n"
            f"sysconfig.get_paths = lambda: {{'include': {str(tmp_path)!r}}}\n"
            "from moe_decode_layer_sm_b200 import build\n"
            "assert not build.can_build_call() and build.build() == build.SO")
    assert r.returncode == 0, r.stderr


def test_a_missing_call_module_is_named():
    r = run("import sys; sys.modules['moe_decode_layer_sm_b200._call'] = None\n"
            "from moe_decode_layer_sm_b200 import attn\n"
            "attn._lib()")
    assert r.returncode != 0 and "_call.so is missing" in r.stderr, r.stderr
