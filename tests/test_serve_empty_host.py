"""A batch without requests: taken, and nothing is launched (no GPU needed)."""
import pytest

from test_serve_host import FAKE, cache, fill, kb, prompts, refused, shared  # noqa: F401 (kb: a fixture)


@pytest.mark.parametrize("first", [None, FAKE])
@pytest.mark.parametrize("total", [0, 100])
def test_no_requests(kb, first, total):  # noqa: F811
    fill(kb, n=0, total=total, shape=(0, 128, 128), c=cache(kb, first=first))
    prompts(kb, n=0, total=total, ws=None, ws_B=0)
    shared(kb, batch=0, q=None, out=None, lse=None, cshape=(0, 128, 128), c=cache(kb, first=first), ws=None, ws_B=0)


def test_first_is_needed_where_there_are_prompts(kb):  # noqa: F811
    refused(kb, kb.EINVAL, fill, c=cache(kb, first=None))
