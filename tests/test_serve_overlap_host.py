"""What kvq_fill_prompts writes must not overlap what it reads (no GPU needed)."""
import pytest

from test_serve_host import FAKE, cache, fill, kb, refused  # noqa: F401 (kb: a fixture)

K, V, STARTS, ELSEWHERE = FAKE << 9, FAKE << 10, FAKE, FAKE << 11
BUFFERS = ("k_codes", "k_scale", "k_zero", "k_resid", "v_codes", "v_scale", "v_zero", "v_resid", "first")


@pytest.mark.parametrize("name", BUFFERS)
def test_over_an_input(kb, name):  # noqa: F811
    """100 tokens of 2 heads, 3 prompts: over the first bytes of an input, or the last 16 of k or v."""
    last = 100 * 256 * 2 - 16
    wide = FAKE << 1                             # beyond every buffer's size
    for at in (K, K + last, V, V + last, STARTS):
        refused(kb, kb.EINVAL, fill, c=cache(kb, at=ELSEWHERE, **{"first": ELSEWHERE + wide, name: at}))


def test_starts_end_where_they_do(kb):  # noqa: F811
    """starts of 4 numbers, and first of 6 right before it: the last of them overlaps, one number earlier it does not (and the
    next check refuses the call)."""
    refused(kb, kb.EINVAL, fill, c=cache(kb, at=ELSEWHERE, first=STARTS - 20))
    refused(kb, kb.EINVAL, fill, c=cache(kb, at=ELSEWHERE, first=STARTS + 12))
    for first in (STARTS - 24, STARTS + 16):
        with pytest.raises(kb.KvqError) as e:
            fill(kb, c=cache(kb, at=ELSEWHERE, first=first, v_resid=V))
        assert "buffers" in str(e.value)
