"""The attention layer's refusals and host arithmetic at the ends of their ranges; no GPU."""
import pytest

from test_ops_layer_abi import P, gdr  # noqa: F401


@pytest.mark.parametrize("D,HQ,HK", [(2**31 - 1, 1, 0), (2**16, 2**15 - 1, 1), (2**31 - 4096, 0, 1), (1, 2**31 - 2, 1)])
def test_rope_refuses_tokens_whose_count_of_units_passes_32_bits(gdr, D, HQ, HK):
    # a thread's next unit is up to 2048 past the last one
    status = gdr.load().rope_turn(0, P(), D, D, HQ, P(2), D, D, P(3), D, D, HK, P(4), D, D, 1, D, 0, P(5), P(6), 0, None, 0, 0, 1.0, 0, None)
    assert status == gdr.GDR_INVALID_ARG


def test_workspace_sizes_past_32_bits(gdr):
    # as attn_fwd takes them: a window past 2^31 sees everything, other sizes are refused, none is cut to 32 bits
    want = gdr.attn_workspace_bytes(1, 65536, 32, 8, 128, [0, 1], [0, 65536])
    for window in (2**31 - 1, 2**31, 2**32 + 5, 2**40):
        assert gdr.attn_workspace_bytes(1, 65536, 32, 8, 128, [0, 1], [0, 65536], window=window) == want, window
    for call in (lambda: gdr.attn_workspace_bytes(11, 11, 2, 2, 64, [0, 11], window=-2**32 + 5), lambda: gdr.attn_workspace_bytes(11, 11, 2**32 + 2, 2, 64, [0, 11]),
                 lambda: gdr.attn_workspace_bytes(11, 11, 2, 2**32 + 2, 64, [0, 11]), lambda: gdr.attn_workspace_bytes(11, 11, 2, 2, 2**32 + 64, [0, 11]),
                 lambda: gdr.lnorm_workspace_bytes(2**32 + 64)):
        with pytest.raises(ValueError):
            call()


def test_workspace_sizes_of_other_documents(gdr):
    # host arrays of another length would be read past their end
    for cu, keys in (([0, 5, 11], [0, 11]), ([0, 11], [0, 5, 11]), ([0, 11], [[0, 11]]), ([], None)):
        with pytest.raises(ValueError, match="cu_"):
            gdr.attn_workspace_bytes(11, 11, 2, 2, 64, cu, keys)


def test_one_long_document_among_many_short_ones_is_cut(gdr):
    # 80 single tokens of 8 key heads are 640 blocks, of which those of one sequence of 65536 keys are
    # as long as 60 of the others: the plan goes by the longest block against an even share, not by
    # the number of blocks
    keys = [0, 65536]
    for _ in range(79):
        keys.append(keys[-1] + 1000)
    fwd, _ = gdr.attn_workspace_bytes(80, keys[-1], 32, 8, 128, list(range(81)), keys)
    assert fwd >= 2 * 80 * 32 * 129 * 4
    even = [1000 * i for i in range(81)]
    assert gdr.attn_workspace_bytes(80, 80000, 32, 8, 128, list(range(81)), even)[0] == 0


def test_outputs_that_are_one_tensor(gdr):
    # one would be written over the other
    lib, bad = gdr.load(), gdr.GDR_INVALID_ARG
    assert lib.lnorm_fwd(0, 3, 1, 64, P(), 64, 64, P(2), 64, 64, 0.5, P(3), None, 0, 1e-5, P(4), P(4), None) == bad
    assert lib.lnorm_bwd(0, 3, 1, 64, P(), 64, 64, P(2), 64, 64, 0.5, P(3), 0, 1e-5, None, 0, 0, P(4), 64, 64, P(5), P(5), None, None, P(6), 1 << 30, None) == bad
    for q, qo, k, ko in ((1, 3, 2, 3), (1, 2, 2, 4), (1, 3, 2, 1), (1, 2, 2, 1)):
        status = lib.rope_turn(0, P(q), 128, 64, 2, P(qo), 128, 64, P(k), 64, 64, 1, P(ko), 64, 64, 4, 64, 64, P(7), P(8), 0, None, 0, 0, 1.0, 0, None)
        assert status == bad, (q, qo, k, ko)
