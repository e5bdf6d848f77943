"""The decoder-attention example runs its stages, and each is as near to the definition as a bf16 output is."""
from __future__ import annotations

import importlib.util
import os

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
def test_decoder_attention(fmt):
    spec = importlib.util.spec_from_file_location("decoder_attention", os.path.join(ROOT, "examples", "decoder_attention.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    errors = example.main(["--format", fmt])
    assert len(errors) == 4
    # rounding to bf16 is 2^-9 at most, 2^-10 on the quadratic mean; the weights' f16 adds less than 2^-11
    assert all(e < 2.0 ** -8 for e in errors.values()), errors
