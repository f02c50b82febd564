"""attention of many rows gives up when the tensor cores do not answer within its limit: it reports that, ends, and leaves
the GPU as it was."""
import pytest
import torch

import kvtest as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,group,n_q,length", [(1, 17, 1, 40), (2, 6, 5, 700), (2, 8, 32, 3000), (8, 4, 64, 3000)])
def test_gives_up_and_reports(heads, group, n_q, length):
    import lattice_entropy_coded_b200 as hq
    a, b = T.pair(heads, [256] * (length // 256) + [length % 256], "E8")
    q = torch.randn(n_q, heads * group, 128, device="cuda").to(torch.bfloat16)
    at = hq.KVAttention(a, b, group)
    want = at(q, torch.empty(n_q, heads * group, 128, device="cuda"))
    torch.cuda.synchronize()
    hq.hq_debug_set_spin_limit(1)
    try:
        for _ in range(20):
            buf = torch.full((n_q, heads * group, 256), 7.0, device="cuda")
            at(q, buf[..., :128])
            torch.cuda.synchronize()
            assert bool((buf[..., 128:] == 7).all())
    finally:
        hq.hq_debug_set_spin_limit(0)
    for c in (a, b):
        assert hq.read_stats(c.stats)["status"] == hq.HQ_ST_TIMEOUT
        c.stats.zero_()
    for _ in range(3):      # every CTA gets its TMEM, and the same bits come out
        assert torch.equal(at(q, torch.empty(n_q, heads * group, 128, device="cuda")), want)
    for c in (a, b):
        assert hq.read_stats(c.stats)["status"] == 0
