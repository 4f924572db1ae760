"""The compiled part of the Python binding (_calls.so): only the 8-bit calls need
it.  CPU only."""
import os
import subprocess
import sys

import pytest

from expanded_rank_matrix_b200 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys
sys.modules['expanded_rank_matrix_b200._calls'] = None  # (importing it fails)
import torch
from expanded_rank_matrix_b200 import externd as X
assert X.load().externd_rank(10, 3, 1.0) == 3 and X.rank(256, 256, 2.0) == 512
assert X.code_words(129) == 16
for call in (lambda: X.quantize_rows(torch.zeros(1, 4)), lambda: X.matmul_i8(None, W, None),
             lambda: X.apply_i8(c, None)):
    class W: q = scale = None
    class c: codes_B = codes_C = D = bound = n = None
    try:
        call()
    except RuntimeError as e:
        assert '_calls' in str(e) and isinstance(e.__cause__, ImportError), e
        assert str(e.__cause__) in str(e), e
    else:
        raise AssertionError('no error')
print('loaded')
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def test_library_loads_without_the_module():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "loaded" in r.stdout, r.stderr[-2000:]


def test_module_is_bound_when_it_is_there():
    import torch

    from expanded_rank_matrix_b200 import externd as X
    with pytest.raises(ValueError, match="CUDA"):
        X.quantize_rows(torch.zeros(1, 4))


def test_another_torch_makes_the_module_stale(monkeypatch):
    """The module is bound to the C++ interface of one torch (and of one Python)."""
    assert not B._stale_calls()
    monkeypatch.setattr(B, "_interfaces", lambda: "another torch")
    assert B._stale_calls()
    monkeypatch.undo()
    assert not B._stale_calls()
    import torch
    assert torch.__version__ in B._interfaces()
