"""What the package's import needs: neither the compiled binding nor torch, as
long as no paged call is made."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "sparse_selected_attention_gb300"


def child(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=600)


def test_star_without_the_binding():
    r = child(f"""
import sys
sys.modules["{PKG}._paged_binding"] = None
from {PKG} import *
assert callable(qsa_prep) and callable(qsa_attn) and callable(qsa_paged_attn)
import torch
z = torch.zeros(1, dtype=torch.int32)
for call in (lambda: qsa_paged_gather(z, z, z, z, z, z, z), lambda: qsa_paged_attn(*[z] * 9), lambda: qsa_paged_prep(*[z] * 10),
             lambda: qsa_page_update(*[z] * 14), lambda: qsa_page_compact(*[z] * 11)):
    try:
        call()
    except RuntimeError as e:
        assert "{PKG}.build" in str(e), e
    else:
        raise SystemExit("a paged call went on without its binding")
""")
    assert r.returncode == 0, r.stderr


def test_star_without_torch():
    r = child(f"""
import sys
sys.modules["torch"] = None
from {PKG} import *
assert callable(qsa_prep) and "qsa_paged_attn" not in globals()
from {PKG} import build
""")
    assert r.returncode == 0, r.stderr


def test_star_with_a_torch_without_cuda():
    r = child(f"""
import sys, torch
sys.modules["{PKG}._paged_binding"] = None
for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, n):
        delattr(torch._C, n)
from {PKG} import *
assert callable(qsa_prep) and callable(qsa_paged_attn)
""")
    assert r.returncode == 0, r.stderr


def test_import_beside_a_stand_in_for_torch():
    """A module put in torch's place, which the import system did not find."""
    r = child(f"""
import sys, types
sys.modules["torch"] = types.ModuleType("torch")
import {PKG} as p
assert callable(p.qsa_prep) and "qsa_paged_attn" in p.__all__
""")
    assert r.returncode == 0, r.stderr


def test_star_has_everything():
    r = child(f"""
import {PKG} as p
from {PKG} import *
assert all(globals()[n] is getattr(p, n) for n in p.__all__) and callable(qsa_page_compact)
assert set(p._PAGED) <= set(p.__all__)
""")
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("name", ["qsa_paged_attn_workspace_bytes", "qsa_pages_workspace_bytes"])
def test_sizes_need_no_binding(name):
    from sparse_selected_attention_gb300 import build
    build.build()
    r = child(f"""
import sys
sys.modules["{PKG}._paged_binding"] = None
import {PKG} as p
assert p.{name}(8, 2) > 0
""")
    assert r.returncode == 0, r.stderr
