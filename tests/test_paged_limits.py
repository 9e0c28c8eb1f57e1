"""Host side of the calls on pages (no GPU): counts at the end of what they are held in."""
import pytest

from test_serving_host import A


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import build
    build.build()
    from rotated_quantized_kv_gb300 import tq as T
    return T


@pytest.mark.parametrize("batch", [(1 << 30) + 1, (1 << 31) - 1])
def test_sequences_past_32_bits(tq, batch):
    """Rounded up to a CTA's share these are no 32-bit numbers: the loop over them would not end."""
    assert tq._lib.tq_page_tables(batch, 16, 4, 8, A, 4, A, A, 3, A, A, A, A, A, None) == -2
    assert tq._lib.tq_page_release(batch, 16, 4, 8, A, 4, A, A, A, A, None) == -2
