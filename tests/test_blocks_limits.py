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
