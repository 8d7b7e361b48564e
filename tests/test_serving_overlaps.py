"""What the calls around the cache write may not share memory with the lists they read by
(lengths, offsets, block table, positions, slots) nor with the status word (no GPU: each call
fails before a launch)."""

import pytest

from bit_quantization_head_b200 import kvtc
from tests.test_serving_refusals import EINVAL, addr, append, cache, cross, decode, desc, rope

C = kvtc.C


@pytest.mark.parametrize("call", [decode, cross])
@pytest.mark.parametrize("written", ["out", "ws"])
def test_attention_refuses_outputs_over_its_lists(call, written):
    at = addr(30)
    # 3 sequences: 12 bytes of lengths, 16 of offsets, 96 of the table; the last bytes count
    assert call(**{written: at}, lens=at + 8) == EINVAL
    assert call(cache(block_table=at + 16), **{written: at}) == EINVAL
    assert call(cache(block_table=at - 92), **{written: at}) == EINVAL
    assert call(cache(status=at + 12), **{written: at}) == EINVAL
    if call is cross:
        assert call(**{written: at}, cu=at + 16) == EINVAL
        assert call(**{written: at}, cu=at - 12) == EINVAL


@pytest.mark.parametrize("call", [decode, cross])
def test_attention_refuses_a_status_word_inside_another_buffer(call):
    for place in (addr(0) + 64, addr(1) + 8, addr(20) + 128, addr(21) + 92):
        assert call(cache(status=place)) == EINVAL


def test_rope_refuses_outputs_over_its_positions():
    # 8 positions of two axes: 64 bytes
    d = desc((32, 32))
    for change in (dict(qo=addr(3), pos=addr(3) + 16), dict(qo=addr(3), pos=addr(3) - 60), dict(ko=addr(4), pos=addr(4) + 32)):
        assert rope(d, **change) == EINVAL


def test_append_refuses_rows_and_pages_over_its_lists():
    d = C.byref(desc())
    for change in (dict(pos=addr(5) + 16), dict(slots=addr(5) + 8), dict(slots=addr(5) - 56), dict(pos=addr(20) + 4096),
                   dict(slots=addr(20) + 4096)):
        assert append(d=d, **change) == EINVAL
    assert append(d=None, q=None, qh=0, qo=None, slots=addr(20) + 4096) == EINVAL
    for place in (addr(20) + 8, addr(2) + 60, addr(3) + 28, addr(5) + 4, addr(0) + 4, addr(1) + 4, addr(4) + 4):
        assert append(cache(status=place), d=d) == EINVAL
