"""owq_gated_plan, the gated block's launch shapes, on the host (no GPU needed): what holds for any
sensible plan, and that the GPU cases reach every kind of launch on a B200."""
import itertools

import pytest

from tests.test_abi import owq  # noqa: F401  (module fixture: builds and loads the library)

SMS = 148   # B200
PRODUCTS = (0, 1, 2)


def _plan(owq, N, K, M, product, sms=SMS):
    st, p = owq.owq_gated_plan(N, K, M, sms, product)
    assert st == 0, (N, K, M, product, sms)
    return p


def test_errors(owq):
    call = owq.owq_gated_plan
    assert (owq.OWQ_GATED_FORWARD, owq.OWQ_GATED_INPUT_GRAD, owq.OWQ_GATED_BACKWARD) == PRODUCTS
    assert call(0, 128, 1, SMS, 0)[0] == 2 and call((1 << 20) + 1, 128, 1, SMS, 0)[0] == 2
    assert call(128, 100, 1, SMS, 0)[0] == 2 and call(128, 0, 1, SMS, 0)[0] == 2 and call(128, 65536 + 128, 1, SMS, 0)[0] == 2
    assert call(128, 128, 0, SMS, 0)[0] == 2 and call(128, 128, 65537, SMS, 0)[0] == 2
    assert call(128, 128, 1, 0, 0)[0] == 12
    assert call(128, 128, 1, SMS, -1)[0] == 12 and call(128, 128, 1, SMS, 3)[0] == 12
    assert owq.LIB.owq_gated_plan(128, 128, 1, SMS, 0, None) == 1


@pytest.mark.parametrize("product", PRODUCTS)
@pytest.mark.parametrize("N,K", [(1, 128), (128, 128), (4096, 4096), (5120, 13824), (13824, 5120), (11008, 4096), (5461, 2048),
                                 (2101, 19456), (1 << 20, 128), (40, 65536)])
def test_invariants(owq, N, K, product):
    for M, sms in itertools.product((1, 17, 32, 33, 64, 65, 100, 128, 129, 192, 193, 256, 257, 300, 1000, 2048, 65536), (1, 2, 16, 132, 148)):
        p = _plan(owq, N, K, M, product, sms)
        rows = 2 * M if product == 2 and M <= 32 else M   # the backward pass of few tokens: two rows a token
        across, steps = (-(-N // 128), K // 128) if product == 0 else (-(-(K // 128) // 2), 2 * -(-N // 128))
        assert p["tile_tokens"] in (64, 128, 192, 256)
        assert p["tile_tokens"] == 64 or rows > p["tile_tokens"] - 64   # no narrower tile holds them all
        assert p["tiles"] == across * -(-rows // p["tile_tokens"])
        pairs = max(1, sms // 2)
        if p["splits"] == 1:
            assert p["whole"] == p["tiles"] and p["steps"] == steps
            continue
        tail = p["tiles"] - p["whole"]
        assert p["whole"] % pairs == 0 and 0 < tail < pairs and tail * p["splits"] <= pairs
        assert p["steps"] >= 4 and -(-steps // p["steps"]) == p["splits"] > 1   # every part holds steps


def _kind(p):
    return "whole" if p["splits"] == 1 else "split" if p["whole"] == 0 else "tail"


@pytest.mark.parametrize("product", (0, 1))
def test_the_gpu_cases_reach_every_kind_of_launch(owq, product):
    from tests.test_gpu_gated_plans import CASES
    got = set()
    for shape, M in CASES:
        p = _plan(owq, *shape[:2], M, product)
        got.add((p["tile_tokens"], _kind(p)))
    assert got == set(itertools.product((64, 128, 192, 256), ("whole", "split", "tail")))


def test_the_gpu_cases_reach_every_backward_of_few_tokens(owq):
    """Two rows a token: whole, split and tail launches, of both products."""
    from tests.test_gpu_gated_plans import CASES
    few = [(s, M) for s, M in CASES if M <= 32]
    for product in (0, 2):
        assert {_kind(_plan(owq, *s[:2], M, product)) for s, M in few} == {"whole", "split", "tail"}


def test_full_size_pair(owq):
    """11008 x 4096: 86 row tiles on 74 pairs, the last 12 split over K; 16 column tiles, all split."""
    for M in (64, 256):
        assert _kind(_plan(owq, 11008, 4096, M, 0)) == "tail"
        assert _kind(_plan(owq, 11008, 4096, M, 1)) == "split"
