"""The buffers that let rows be taken back from the 8-bit cache: the C ABI's checks, with made-up
pointers (nothing is launched)."""

import pytest
import torch

from test_kv8_refusals import A, ALIGN, EVERY, NULL, UNSUPPORTED, cache

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: host checks only")
NAMES = ("k_last", "v_last", "blocks")


@pytest.mark.parametrize("call", EVERY)
def test_all_or_none(call):
    assert call(c=cache(**{n: None for n in NAMES})) == UNSUPPORTED
    for name in NAMES:
        assert call(c=cache(**{name: None})) == NULL
        assert call(c=cache(**{n: None for n in NAMES if n != name})) == NULL


@pytest.mark.parametrize("call", EVERY)
def test_alignment(call):
    assert call(c=cache(k_last=A + 8)) == ALIGN and call(c=cache(v_last=A + 8)) == ALIGN
    assert call(c=cache(blocks=A + 4)) == ALIGN
    assert call(c=cache(blocks=A + 8)) == UNSUPPORTED
