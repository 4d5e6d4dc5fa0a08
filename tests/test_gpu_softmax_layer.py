"""The example layer (examples/softmax_layer.py): prompts then single tokens equal the same tokens at once, and
continuations behind shared rows equal separate sequences."""
import importlib.util
import os

import pytest

from gpu_util import ensure_built, require_gpu

pytestmark = pytest.mark.gpu


def test_prompts_tokens_and_shared_rows_agree():
    ensure_built()
    require_gpu()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "softmax_layer.py")
    spec = importlib.util.spec_from_file_location("softmax_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    example.main()
