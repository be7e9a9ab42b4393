"""Which form of the windowed forward runs (attn_window_fwd_form): tests that
mean one of them get it on the device at hand, and would say so if the rule that
picks it moved away from their sizes."""

import pytest

import long_context_causal_blockwise_gb300 as lcb
import test_gpu_window
import test_gpu_window_rows

form = lcb.attn_window_fwd_form


def _cases(test):
    """The cases that a test is parametrised with."""
    return [tuple(c) for m in test.pytestmark if m.name == "parametrize" for c in m.args[1]]


@pytest.mark.gpu
def test_cases_reach_the_form_that_they_are_for():
    for B, H, Hkv, Sq, Sk, window, sinks, pos0 in _cases(test_gpu_window.test_forward_in_128_row_tiles):
        n = 608 // (B * Hkv * ((Sq * (H // Hkv) + 15) // 16)) + 1  # as many heads as the test takes
        assert form(B, n * H, n * Hkv, Sq, Sk, window, sinks, pos0) == "tiles", (Sq, Sk)
    for c in _cases(test_gpu_window.test_more_blocks_than_sms) + _cases(test_gpu_window_rows.test_more_than_one_group_of_heads):
        assert form(*c) == "tiles", c
    for c in _cases(test_gpu_window.test_forward_blocks_shared_by_a_cluster):  # one of them says that it is not
        assert form(*c) == ("tiles" if c[7] == -150 else "cluster"), c
    for H, Hkv, Sq in _cases(test_gpu_window.test_few_rows_forward):
        assert form(2, H, Hkv, Sq, 5000, 3000, 4) == "split", (H, Hkv, Sq)
    # of the five cases of several row tiles three are split; the other two are blocks shared by a cluster
    assert [form(1, H, Hkv, Sq, Sk, w, 3) for H, Hkv, Sq, Sk, w in _cases(test_gpu_window.test_forward_split_over_row_tiles)] \
        == ["split", "cluster", "cluster", "split", "split"]
    assert [form(1, H, Hkv, Sq, Sk, w) for H, Hkv, Sq, Sk, w in test_gpu_window_rows.FORMS] == ["split", "cluster", "tiles"]
    assert {form(2, H, Hkv, S, S, 1) for H, Hkv, S in _cases(test_gpu_window.test_row_of_one_key_gives_its_v)} \
        == {"split", "tiles"}


def test_empty_sides_and_refusals():
    """Sizes that launch nothing, and those that the forward refuses; no device needed."""
    assert form(1, 2, 2, 0, 300, 64) == "empty" and form(1, 2, 2, 300, 0, 64) == "empty"
    assert form(1, 2, 2, 8, 300, 64) == "split"  # up to 16 query rows a K/V head, on any device
    for bad in (dict(window=0), dict(sinks=-1), dict(Hkv=3), dict(D=64), dict(q_pos0=1 << 29), dict(B=0), dict(Sq=-1)):
        with pytest.raises(lcb.AttnError):
            form(**{**dict(B=1, H=4, Hkv=2, Sq=40, Sk=300, window=64), **bad})
