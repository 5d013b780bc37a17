"""The 4-bit training and serving example: the loss falls, and serving one
token at a time agrees with the training forward as far as the two
quantisations of the same tokens do."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "fp4_train_and_serve.py")


@pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
def test_train_and_serve(fmt):
    spec = importlib.util.spec_from_file_location("fp4_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    lines = []
    first, last, far = m.main(fmt, say=lines.append)
    assert last < 0.5 * first
    # MXFP4 blocks do not depend on the other tokens: the same bits but for the
    # order of sums; NVFP4 tokens get a tensorwise scale of their own.
    assert far < (0.2 if fmt == 0 else 0.02)
    assert len(lines) > 3
