"""The largest batches that decode attention behind shared prefixes takes. CPU only: nothing is
launched."""
import pytest

from tests.test_abi_serving import UNSUPPORTED, mla

__all__ = ["mla"]

THREADS = 384  # of a CTA that look up pages at the most


def weight(B, rows):
    return B * (-(-rows // 128) + 4)


def rows_for(B, most):
    """The largest bound of a batch's lengths whose weight is at most `most`."""
    return 128 * (most // B - 4)


@pytest.mark.parametrize("B", [1, 127, 128, 3001, 4096])
def test_page_places_stay_in_32_bits(mla, B):  # noqa: F811
    """A thread's place (two for each weight) goes one step of all threads past the last one."""
    size = mla.decode_shared_workspace_size
    limit = 2 ** 30 - 1025
    rows = min(rows_for(B, limit), 2 ** 31 - 1)
    assert 2 * weight(B, rows) + THREADS <= 2 ** 31 - 1
    assert size(B, 1, 16, rows, 1) > mla.WS_HEADER_BYTES
    more = rows + 128
    if more > 2 ** 31 - 1:
        return
    while 2 * weight(B, more) + THREADS <= 2 ** 31 - 1 and weight(B, more) <= limit:
        more += 128
    with pytest.raises(mla.MLAError) as e:
        size(B, 1, 16, more, 1)
    assert e.value.code == UNSUPPORTED


@pytest.mark.parametrize("heads", [16, 128])
def test_a_place_that_would_wrap(mla, heads):  # noqa: F811
    """2^31 - 8 places fit in 32 bits, the threads' next ones do not."""
    assert 2 * weight(127, 1082195968) == 2 ** 31 - 8
    with pytest.raises(mla.MLAError) as e:
        mla.decode_shared_workspace_size(127, 1, heads, 1082195968, 1)
    assert e.value.code == UNSUPPORTED
