"""How long the kernels' waits on barriers last at most, by their source (no GPU needed)."""
import os
import re

from kv_cache_quantization_kvq_gb300 import builder


def source(name):
    with open(os.path.join(builder.CSRC, name), encoding="utf-8") as f:
        return f.read()


def test_waits_are_bounded_in_time():
    """Barriers are polled in two places.  kvq_bulk.cuh's waits, of the quantizers' rings, are for the CTA's own copies and for
    the warps that use them; those of the tensor-core kernels, whose CTAs wait for one another too, are kvq_tc.cuh's: a
    poll lasts 1 us at most, and they run out after some seconds."""
    polled = {f for f in os.listdir(builder.CSRC) if re.search(r"mbarrier\.(try|test)_wait", source(f))}
    assert polled == {"kvq_bulk.cuh", "kvq_tc.cuh"}
    tc = source("kvq_tc.cuh")
    polls = 1 << int(re.search(r"kPolls = 1u << (\d+);", tc).group(1))
    hints = re.findall(r"try_wait\.parity\.shared::cta\.b64 p, \[%1\], %2(?:, (\d+))?;", tc)
    assert len(hints) == len(re.findall(r"mbarrier\.(?:try|test)_wait", tc)) > 0
    assert all(h and polls * int(h) * 1e-9 < 5.0 for h in hints)
