"""Host checks of the block operators at the ends of what they take: long
windows, memory that overlaps.  None of this launches anything."""
import pytest

from test_blocks_host import K, P, Handle  # noqa: F401  (K is a fixture)


@pytest.mark.parametrize("R", [32, 4096, 16288, 16320, 16384, 32768, 65440])
def test_workspace_holds_every_split(K, R):
    """A tail of R + 31 tokens is shared out 64 tokens a split, and a packed
    split lies beside it: the workspace has slots for all of them, and for
    their groups of sixteen."""
    splits = (R + 31 + 63) // 64 + 1
    with Handle(K, batch=1, n_kv_heads=1, n_q_heads=1, residual=R, max_tokens=4 * R, length=3 * R + 31) as h:
        slot = 8 * (128 + 2) * 4  # of a split or a group: outputs, max and sum of eight heads
        assert K.kivi_block_workspace_bytes(h) >= (splits + -(-splits // 16)) * slot


def test_longer_windows_are_refused(K):
    """More splits than two levels of merges take."""
    lib, R = K.lib(), 65472
    with Handle(K, residual=R, max_tokens=2 * R, length=2 * R) as h:
        ws, rec = K.kivi_block_workspace_bytes(h), K.kivi_block_records_bytes(h)
        assert lib.kivi_decode_attention_blocks(h, P, 1, P, 4, P, 0.0, P, ws, None) == K.KIVI_ESHAPE
        assert lib.kivi_decode_attention_topk(h, P, 1, 4, 0, 0, P, 4092, P, P, 0.0, P, ws, None) == K.KIVI_ESHAPE
        assert lib.kivi_decode_attention_mass(h, P, 1, P, 0.0, P, P, 4092, 1.0, P, ws, P, rec, None) == K.KIVI_ESHAPE


def test_rows_that_overlap_are_refused(K):
    """A result may take its source's place whole; any other overlap would have
    one unit's rows written while another's are read."""
    lib = K.lib()
    with Handle(K, length=4000) as h, Handle(K, base=1 << 34) as into:  # 2 x 4 units, 124 blocks
        Q = 1 << 28
        ws, rec = K.kivi_block_workspace_bytes(h), K.kivi_block_records_bytes(h)
        bytes_of = lambda n: 4 * 8 * n  # noqa: E731
        free = lib.kivi_select_blocks(h, Q, 124, 4, 0, 0, 2 * Q, None)  # what a call gets that passes every check
        inside = (0, 4, bytes_of(124) - 4)
        for at in inside:
            assert lib.kivi_select_blocks(h, Q, 124, 4, 0, 0, Q + at, None) == K.KIVI_EINVAL
            assert lib.kivi_decode_attention_topk(h, P, 1, 4, 0, 0, Q, 124, Q + at, P, 0.0, P, ws, None) == K.KIVI_EINVAL
        assert lib.kivi_select_blocks(h, Q, 124, 4, 0, 0, Q + bytes_of(124), None) == free
        assert lib.kivi_select_blocks(h, Q, 124, 4, 0, 0, Q - bytes_of(4), None) == free
        assert lib.kivi_select_blocks(h, Q, 124, 4, 0, 0, Q - bytes_of(4) + 4, None) == K.KIVI_EINVAL

        def mass(a, b):
            return lib.kivi_decode_attention_mass(h, P, 1, P, 0.0, a, b, 125, 1.0, P, ws, P, rec, None)
        for a, b in ((Q, Q + 4), (Q + 4, Q), (Q, Q + bytes_of(125) - 4), (Q + 4 * 125, Q)):
            assert mass(a, b) == K.KIVI_EINVAL
        assert mass(Q, Q) == mass(Q, Q + bytes_of(125)) == mass(None, Q) == free

        def evict(m, kept, out, to=into, out_row=125):
            return lib.kivi_evict_blocks(h, to, m, 125, 20, 0, 0, kept, 20, out, out_row, None)
        for to in (into, h):
            for m, kept, out in ((Q, Q, None), (Q, Q + bytes_of(125) - 4, 2 * Q), (Q, 2 * Q, 2 * Q + 4 * 20), (Q, 2 * Q, Q + 4),
                                 (Q + 4 * 125, 2 * Q, Q)):
                assert evict(m, kept, out, to) == K.KIVI_EINVAL
            assert evict(Q, 2 * Q, Q, to) == evict(Q, 2 * Q, 3 * Q, to) == evict(Q, 2 * Q, None, to) == free
            assert evict(Q, Q + bytes_of(125), Q + bytes_of(125 + 20), to) == free
        assert K.kivi_cache_length(h) == 4000 and K.kivi_cache_length(into) == 0


def test_whole_attention_over_too_many_splits_is_refused(K):
    """The whole-cache attention merges 256 splits: a window of 64 tokens a
    split without a packed tile behind it has no other plan."""
    lib, R = K.lib(), 32768
    for length, refused in ((16384, False), (16385, True), (30000, True), (R + 31, True), (2 * R + 40, False)):
        with Handle(K, residual=R, max_tokens=4 * R, length=length) as h:
            assert (K.kivi_attention_splits(h, length) > 256) == refused
            ws = K.kivi_attention_workspace_bytes(h)
            got = [lib.kivi_decode_attention(h, P, 1, P, 0.0, P, ws, None),
                   lib.kivi_decode_step(h, P, P, 1, P, 1, P, 0.0, P, ws, None)]
            # (16384 tokens: the step's token is one too many)
            assert got[0] == K.KIVI_ESHAPE if refused else got[0] != K.KIVI_ESHAPE
            assert got[1] == K.KIVI_ESHAPE if refused and length != R + 31 or length == 16384 else got[1] != K.KIVI_ESHAPE
            assert K.kivi_cache_length(h) == length
            K.kivi_set_attention_splits(h, 1000)
            if K.kivi_attention_splits(h, length) > 256:
                assert lib.kivi_decode_attention(h, P, 1, P, 0.0, P, ws, None) == K.KIVI_ESHAPE
