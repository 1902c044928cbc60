"""Workspace sizes of kvq_attend_shared and kvq_attend_prompts, over every form (no GPU needed)."""
import pytest

from test_serve_host import FAKE, cache, kb, kq, prompts, refused, shared, vq  # noqa: F401 (kb: a fixture)

# query rows of a KV head on both sides of every form's ends, as (batch, group, n)
ROWS = [(1, 1, 1), (2, 4, 1), (9, 1, 1), (4, 4, 1), (17, 1, 1), (8, 4, 1), (11, 3, 1), (16, 8, 1), (129, 1, 1), (64, 4, 1),
        (257, 1, 1), (128, 4, 1), (57, 9, 1), (256, 8, 1), (683, 3, 1), (1, 4, 9), (4, 4, 33), (2, 64, 20)]


@pytest.mark.parametrize("C", [64, 128])
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("batch,group,n", ROWS)
def test_shared(kb, C, own, batch, group, n):  # noqa: F811
    """A longer store or buffer never needs less, and a call with less than the query's bytes is refused."""
    def size(T, R, To, Ro):
        return kb.kvq_attend_shared_workspace((2, T, C), R, (2 * batch, To, C) if own else None, Ro if own else 0, batch, n, group)

    lengths = (0, 64, 1024, 2048, 2112, 8192, 65536, 1 << 20)
    for other in ((64, 64), (8192, 64)):
        last = 0
        for T in lengths:
            have = size(T, 64, *other)
            assert have > 0 and have >= last and size(T, 4096, *other) >= have
            last = have
        if own:
            last = 0
            for T in lengths:
                have = size(*other, T, 64)
                assert have >= last and size(*other, T, 4096) >= have
                last = have
    want = size(128, 64, 128, 64)
    kw = dict(batch=batch, n=n, group=group, shape=(2, 128, C), cshape=(2 * batch, 128, C), q=1 << 40, out=1 << 41, lse=1 << 42)
    if not own:
        kw["c"] = None
    refused(kb, kb.EWORKSPACE, shared, ws=None, **kw)
    refused(kb, kb.EWORKSPACE, shared, ws_B=want - 1, **kw)
    refused(kb, kb.EINVAL, shared, ws=FAKE + 16, ws_B=want, **kw)


@pytest.mark.parametrize("total", [1, 100, 70000])
@pytest.mark.parametrize("group", [1, 3, 64])
def test_prompts(kb, group, total):  # noqa: F811
    want = kb.kvq_attend_prompts_workspace(3, total, group, 2, 128)
    assert want > 0 and kb.kvq_attend_prompts_workspace(3, total + 1000, group, 2, 128) > want
    assert kb.kvq_attend_prompts_workspace(3 + 1000, total, group, 2, 128) >= want
    kw = dict(n=3, total=total, group=group, qs=2 * group * 128, q=1 << 40, k=1 << 41, v=1 << 42, out=1 << 43, lse=1 << 44)
    refused(kb, kb.EWORKSPACE, prompts, ws=None, **kw)
    refused(kb, kb.EWORKSPACE, prompts, ws_B=want - 1, **kw)
    refused(kb, kb.EINVAL, prompts, ws=FAKE + 16, ws_B=want, **kw)
