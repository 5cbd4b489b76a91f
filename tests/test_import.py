"""The package where its library is not built: every name is there, and a call says what is
missing."""
import os
import shutil
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "row_wise_normalization_gb300"

PROGRAM = """
from row_wise_normalization_gb300 import *
import row_wise_normalization_gb300 as rn
import torch
assert embed_fwd is rn.embed_fwd and all(callable(f) for f in (ln_fwd, embed_bwd, logprob_bwd))
try:
    rn.capi.embed_bwd_workspace_size(1, 1, 1)
except RuntimeError as e:
    assert "not built" in str(e)
else:
    raise SystemExit("a library was found")
from row_wise_normalization_gb300 import tokens
try:
    tokens._C.embed_fwd
except RuntimeError as e:
    assert "not built" in str(e)
else:
    raise SystemExit("a library was found")
print("fine")
"""


def test_star_import_without_the_library(tmp_path):
    (tmp_path / PKG).mkdir()
    for f in ("__init__.py", "capi.py", "tokens.py"):
        shutil.copy(os.path.join(ROOT, PKG, f), tmp_path / PKG / f)
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=tmp_path, capture_output=True,
                       text=True, env={**os.environ, "PYTHONPATH": ""})
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stdout + r.stderr
