"""How the decayed linear attention cuts its problems into segments, read off
the workspace that a call asks for: one state for each segment of each head."""

import ctypes

import pytest

from token_level_head_phi_gb300 import binding as mb
from token_level_head_phi_gb300 import build as mbuild


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mb.load()


def segments(lib, batch, heads, tokens, key_dim, value_dim, dtype):
    p, n = mb.MhlaDecayParams(), ctypes.c_size_t(0)
    p.batch, p.heads, p.tokens, p.key_dim, p.value_dim = batch, heads, tokens, key_dim, value_dim
    p.dtype, p.scale = mb.DTYPES[dtype], 1.0
    assert lib.mhla_decay_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == mb.MHLA_OK
    return max(1, n.value // (4 * batch * heads * key_dim * value_dim))


@pytest.mark.parametrize("heads,tokens", [(60, 2048), (64, 2048), (76, 4096)])
def test_float32_rows_of_128_fill_the_sms_with_one_segment(lib, heads, tokens):
    """One CTA of those rows fits an SM: two slices of each head are a wave, more segments only wait."""
    assert segments(lib, 1, heads, tokens, 128, 128, "f32") == 1
