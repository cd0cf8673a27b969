"""The turns of the products' epilogue buffers, modelled on the CPU.

A warp of the 16-bit products' epilogue writes its 32 x 32 pieces into two shared-memory buffers in turn.  A
whole piece leaves by an asynchronous bulk store, which goes on reading its buffer; the last rows of a segment
are copied out by the lanes.  Before a buffer is written again the warp waits until at most the newest bulk
group is still being read (csrc/dense_epilogue.cuh, store_piece32; csrc/dense.cu, store_piece), which is enough
only if every piece commits one group, also one that leaves no store behind.  This test restates that protocol
and checks, over every order of whole and partial pieces, that no buffer is written while a store may still read
it, and that the check notices the protocol that commits whole pieces only."""
import itertools


def overwritten_while_read(pieces, commit_partial):
    """pieces: True for a whole piece, False for a partial one.  The index of the first piece that is written into
    a buffer a pending store may still read, or None.  Stores are taken to be as slow as the waits allow."""
    groups = []                                  # committed groups not known to be read: (buffer,) or ()
    turn = 0
    for at, whole in enumerate(pieces):
        buffer = turn
        turn ^= 1
        groups = groups[-1:]                     # cp.async.bulk.wait_group.read 1
        if any(buffer in g for g in groups):
            return at
        if whole:
            groups.append((buffer,))
        elif commit_partial:
            groups.append(())
    return None


def test_one_group_a_piece_keeps_the_buffers_apart():
    for n in range(1, 11):
        for pieces in itertools.product((True, False), repeat=n):
            assert overwritten_while_read(pieces, commit_partial=True) is None, pieces


def test_the_model_notices_a_piece_without_a_group():
    assert overwritten_while_read((True, False, True), commit_partial=False) == 2
    assert overwritten_while_read((True, False, False), commit_partial=False) == 2
    # whole pieces alone need nothing more
    assert overwritten_while_read((True,) * 10, commit_partial=False) is None
