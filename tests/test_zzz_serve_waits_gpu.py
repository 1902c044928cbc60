"""No bounded wait gave up in the kernels of serving a batch: each form with waits
is run once, so that this file means something on its own."""
import pytest

from gpu_util import kb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kb()


@pytest.mark.parametrize("C", [64, 128])
@pytest.mark.parametrize("lens", [[300], [200, 900, 5] * 12])      # without a plan and with one
def test_packed_prompts(b, C, lens):
    import torch
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((sum(lens), 12, C), generator=g, device="cuda").bfloat16()
    starts = torch.tensor([0] + lens, dtype=torch.int32, device="cuda").cumsum(0, dtype=torch.int32)
    out, lse = b.attend_prompts(*x.split([8, 2, 2], 1), starts)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert b.kvq_wait_timeouts() == 0


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("C", [64, 128])
@pytest.mark.parametrize("batch", [3, 15, 40, 300])                # rows of warps, of one SM, of pairs, expanded
def test_shared_prefix(b, batch, C, bits):
    import torch
    g = torch.Generator(device="cuda").manual_seed(9)
    kw = dict(scale_dtype=b.BF16, zero_dtype=b.BF16, residual=64)
    kqp, vqp = (b.QParams.asym(bits, 0, 2 ** bits - 1, axis=a, group=64, **kw) for a in (b.ALONG_T, b.ALONG_C))

    def cache(outer, T):
        x = torch.randn((2, outer, T, C), generator=g, device="cuda").bfloat16()
        return b.KVCache.from_quantized(b.quantize(x[0], kqp), b.quantize(x[1], vqp), 2)

    q = torch.randn((batch, 1, 16, C), generator=g, device="cuda").bfloat16()
    out, lse = b.attend_shared(q, cache(2, 2112), cache(2 * batch, 192))
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert b.kvq_wait_timeouts() == 0
