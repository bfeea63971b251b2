"""The example of a whole attention layer, which checks its own steps."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapter_attention.py")


@pytest.mark.parametrize("kw", [{}, dict(adapters=1, per_adapter=1, prompt=16, decode=1)], ids=["default", "one"])
def test_adapter_attention(kw):
    spec = importlib.util.spec_from_file_location("adapter_attention", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.main(**kw)
