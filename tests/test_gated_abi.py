"""The gated block's and the clipping's C calls refuse bad arguments on the host, before any
device use (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def owq():
    from weight_only_mixed_owq_b200 import build
    build.build()
    import weight_only_mixed_owq_b200 as m
    return m


FAKE = 0x10000


def test_gated_calls_want_live_handles(owq):
    for gate, up in ((None, None), (FAKE, None), (None, FAKE), (FAKE, FAKE)):
        assert owq.owq_gated_gemv(gate, up, 0, FAKE, FAKE, 1) == 10
        assert owq.owq_gated_gemm(gate, up, 0, FAKE, FAKE, 64, FAKE, 1 << 20) == 10
        assert owq.owq_gated_grad(gate, up, 0, FAKE, FAKE, FAKE, FAKE, 64, FAKE, 1 << 20) == 10
        assert owq.owq_gated_backward(gate, up, 0, FAKE, FAKE, FAKE, FAKE, FAKE, 64, FAKE, 1 << 20) == 10
        assert owq.owq_gated_input_grad(gate, up, FAKE, FAKE, FAKE, 64, FAKE, 1 << 20) == 10
        assert owq.owq_gated_workspace(gate, up, 64)[0] == 10


def table(owq, *entries):
    return (owq.OwqGrad * max(1, len(entries)))(*[owq.OwqGrad(*e) for e in entries])


F32, F16, BF16 = 0, 1, 2


@pytest.mark.parametrize("status,entries", [
    (12, [(FAKE, FAKE, 4, 3)]),                                    # no such type
    (12, [(FAKE, FAKE, 4, -1)]),
    (2, [(FAKE, FAKE, -1, F32)]),                                  # sizes
    (2, [(FAKE, FAKE, (1 << 38) + 1, F16)]),
    (2, [(FAKE, FAKE, 1 << 38, F32), (FAKE + (1 << 41), FAKE + (1 << 41), 1, F32)]),   # over 1 TB together
    (1, [(None, FAKE, 4, F32)]),
    (1, [(FAKE, None, 4, F32)]),
    (6, [(FAKE + 2, FAKE + 2, 4, F32)]),                           # alignment to the value
    (6, [(FAKE, FAKE + 4096 + 1, 4, F16)]),
    (12, [(FAKE, FAKE + 8, 4, F32)]),                              # an output across its own input
    (12, [(FAKE, FAKE, 4, F32), (FAKE, FAKE, 4, F32)]),            # one tensor twice, in place
    (12, [(FAKE, FAKE, 8, F32), (FAKE + 28, FAKE + 28, 1, F32)]),  # in place inside another
    (12, [(FAKE, FAKE + 4096, 8, BF16), (FAKE + 8192, FAKE + 4096 + 14, 8, BF16)]),   # two outputs that meet
    (12, [(FAKE, FAKE + 4096, 8, F32), (FAKE + 4096, FAKE + 8192, 8, F32)]),          # one's output is the other's input
])
def test_clip_create_refuses(owq, status, entries):
    st, handle = owq.owq_clip_create(table(owq, *entries), len(entries))
    assert st == status and not handle


def test_clip_handles(owq):
    assert owq.owq_clip_create(table(owq), -1)[0] == 2
    assert owq.owq_clip_create(table(owq), (1 << 20) + 1)[0] == 2
    assert owq.owq_clip_create(None, 1)[0] == 1
    assert owq.LIB.owq_clip_create(None, 0, None, None) == 1
    assert owq.owq_clip_grads(None, 1.0, FAKE) == 10 and owq.owq_clip_grads(FAKE, 1.0, FAKE) == 10
    assert owq.owq_clip_free(None) == 0 and owq.owq_clip_free(FAKE) == 10


def test_the_entries_match_the_header(owq):
    """owq_grad_t as C lays it out on this platform."""
    assert ctypes.sizeof(owq.OwqGrad) == 32
    assert [getattr(owq.OwqGrad, n).offset for n, _ in owq.OwqGrad._fields_] == [0, 8, 16, 24]
