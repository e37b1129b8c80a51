"""Loading and building on the CPU: the operators' module works with the library beside it alone,
and the tail needs neither that module nor what builds it."""
import os
import shutil
import subprocess
import sys

import pytest

from latent_moe_layer_route_gb300 import build

ROOT = build.ROOT


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _python(code, *args):
    return subprocess.run([sys.executable, "-c", code, *map(str, args)], cwd=ROOT,
                          capture_output=True, text=True)


def test_a_library_elsewhere_serves_the_tail_and_refuses_the_operators(tmp_path):
    """The operators' module is linked to one copy of the library: a handle made by another copy
    must not reach it."""
    other = tmp_path / "libklt.so"
    shutil.copy(build.LIB_PATH, other)
    r = _python("""
import sys, torch
from latent_moe_layer_route_gb300 import binding as B
assert B.load_library(sys.argv[1]).klt_status(None) == B.KLT_ERR_INVALID_ARG
assert B.strerror(B.KLT_ERR_ALIGN)
w = torch.zeros(256, 256, dtype=torch.uint8)
for call in (lambda: B.quantize_fp8(torch.zeros(4, 256)), lambda: B.BlockNorm(256),
             lambda: B.Fp8Linear(w, torch.ones(2, 2))):
    try:
        call()
    except RuntimeError as e:
        assert "only" in str(e), e
    else:
        raise SystemExit("an operator ran on another copy of the library")
""", other)
    assert r.returncode == 0, r.stdout + r.stderr


def test_the_tail_loads_without_the_operators_module():
    r = _python("""
from latent_moe_layer_route_gb300 import binding as B
B.MARSHAL_PATH += ".absent"
assert B.load_library().klt_status(None) == B.KLT_ERR_INVALID_ARG
import torch
try:
    B.quantize_fp8(torch.zeros(4, 256))
except RuntimeError as e:
    assert "not built" in str(e), e
else:
    raise SystemExit("no error")
""")
    assert r.returncode == 0, r.stdout + r.stderr


def test_a_link_to_the_library_is_the_library(tmp_path):
    link = tmp_path / "libklt.so"
    os.symlink(build.LIB_PATH, link)
    r = _python("""
import sys, torch
from latent_moe_layer_route_gb300 import binding as B
B.load_library(sys.argv[1])
try:
    B.quantize_fp8(torch.zeros(4, 256))
except ValueError as e:  # a host tensor
    assert "CUDA" in str(e), e
""", link)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("broken", ["torch", "compiler"])
def test_the_library_builds_where_the_operators_module_does_not(tmp_path, broken):
    """Without torch, or where the module's compiler fails, build() still makes libklt.so, and no
    module of an earlier build stays beside it."""
    r = _python("""
import os, sys, warnings
from latent_moe_layer_route_gb300 import build as b
out, broken = sys.argv[1:]
b.OUT_DIR, b.LIB_PATH = out, os.path.join(out, "libklt.so")
b.MARSHAL_PATH = os.path.join(out, "_marshal.so")
b.SOURCES = ["klt_noalloc.cu"]  # one of them will do
open(b.MARSHAL_PATH, "w").close()
os.utime(b.MARSHAL_PATH, (0, 0))
if broken == "torch":
    find = b.importlib.util.find_spec
    b.importlib.util.find_spec = lambda name, *a: None if name == "torch" else find(name, *a)
else:
    b._gxx = lambda cmd, what: (_ for _ in ()).throw(RuntimeError("no compiler"))
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    assert b.build() == b.LIB_PATH
assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.MARSHAL_PATH)
assert any("not built" in str(w.message) for w in seen), [str(w.message) for w in seen]
""", tmp_path, broken)
    assert r.returncode == 0, r.stdout + r.stderr


def test_the_modules_object_belongs_to_one_interpreter():
    assert os.path.exists(os.path.join(build.OUT_DIR, "klt_marshal" + build.EXT_SUFFIX + ".o"))
