"""Importing the binding where only a part of it is there: without the compiled
binding of the short calls, and with an earlier build of the library.  What is
there works; a call that needs what is missing says so."""
import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "top_routing_mxfp4_gb300")
LATER = {"lmoe_rms_norm", "lmoe_residual_norm", "lmoe_linear_mxfp4", "lmoe_linear_mxfp4_workspace_size",
         "lmoe_grouped_linear_bf16", "lmoe_grouped_swiglu_bf16", "lmoe_grouped_workspace_size",
         "lmoe_forward_residual_block", "lmoe_residual_block_workspace_size"}


@pytest.fixture(scope="module")
def library():
    from top_routing_mxfp4_gb300 import build
    return build.build()


def _python(code, cwd, **env):
    r = subprocess.run([sys.executable, "-c", code], cwd=cwd, env=dict(os.environ, PYTHONPATH=str(cwd), **env),
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_without_the_compiled_binding(library, tmp_path):
    pkg = tmp_path / "top_routing_mxfp4_gb300"
    pkg.mkdir()
    for f in ("__init__.py", "build.py", "lmoe.py"):
        shutil.copy(os.path.join(PKG, f), pkg / f)
    os.symlink(library, pkg / "liblmoe.so")
    out = _python("""
import torch
from top_routing_mxfp4_gb300 import lmoe
assert lmoe.workspace_size(64, 3584, 896, 16, 512) > 0 and lmoe.linear_mxfp4_workspace_size(64, 256, 96) > 0
x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64)
for _ in range(2):
    for call in (lambda: lmoe.rms_norm(x, w), lambda: lmoe.linear_mxfp4(x, w, w, 4)):
        try:
            call()
        except ImportError as e:
            assert '_lmoe_torch' in str(e) and 'build' in str(e), e
        else:
            raise AssertionError('no refusal')
print(lmoe.version())
""", tmp_path)
    assert "sm_103a" in out


def test_with_an_earlier_library(library, tmp_path):
    """LMOE_LIBRARY selects a library that lacks the later entry points."""
    header = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "lmoe.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(lmoe_[a-z0-9_]+)\s*\(", header)))
    assert LATER <= set(names)
    src = tmp_path / "earlier.c"
    src.write_text('const char *lmoe_version(void) { return "earlier"; }\n' +
                   "".join(f"long {n}(void) {{ return 0; }}\n" for n in names if n not in LATER | {"lmoe_version"}))
    lib = tmp_path / "libearlier.so"
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    out = _python("""
import torch
from top_routing_mxfp4_gb300 import lmoe
x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64)
for call in (lambda: lmoe.rms_norm(x, w), lambda: lmoe.residual_norm(x, x), lambda: lmoe.grouped_workspace_size(),
             lambda: lmoe.linear_mxfp4_workspace_size(4, 64, 64)):
    try:
        call()
    except (ImportError, RuntimeError) as e:
        assert 'lmoe_' in str(e) and 'libearlier.so' in str(e), e
    else:
        raise AssertionError('no refusal')
print(lmoe.version(), lmoe.small_batch_pairs())
""", ROOT, LMOE_LIBRARY=str(lib))
    assert out.split() == ["earlier", "0"]


def test_the_compiled_binding_is_of_this_torch_and_python(library, monkeypatch):
    """It is rebuilt when torch or Python changed under it, whatever the files' times say, and one built for others is
    refused."""
    from top_routing_mxfp4_gb300 import build
    import torch
    assert not build._bind_stale()
    assert torch.__version__ in build._bind_tag() and sys.implementation.cache_tag in build._bind_tag()
    with monkeypatch.context() as m:
        m.setattr(build, "_bind_tag", lambda: "another torch")
        assert build._bind_stale()
    out = _python("""
import torch
torch.__version__ = '0.0.0'
from top_routing_mxfp4_gb300 import lmoe
try:
    lmoe.rms_norm(torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64))
except ImportError as e:
    print(e)
""", ROOT)
    assert "0.0.0" in out and torch.__version__ in out
