"""A tree of one draft, or over one KV head: tensors whose strides differ only in a dimension of one are one layout."""
import pytest
import torch

import kvtest as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,n_q", [(4, 1), (1, 3), (1, 1)])
def test_keys_as_written_and_values_as_a_slice(heads, n_q):
    """The values stay where the projection left them, as the README's step has it; .contiguous() keeps such strides."""
    import lattice_entropy_coded_b200 as hq
    a, b = T.pair(heads, [40], "E8")
    x = torch.randn(n_q, 4 * heads, 128, device="cuda").to(torch.bfloat16)
    q, vd = x[:, :2 * heads], x[:, 3 * heads:].transpose(0, 1)
    kd = x[:, 2 * heads:3 * heads].transpose(0, 1).clone(memory_format=torch.contiguous_format).reshape(heads, n_q, 128)
    if n_q > 1:
        vd = vd.as_strided(vd.shape, (7 * vd.stride(0), vd.stride(1), 1))     # one head: its stride may be anything
        kd = x[:, 2 * heads:3 * heads].transpose(0, 1)
    assert kd.stride() != vd.stride()
    m = torch.tensor([(2 << i) - 1 for i in range(n_q)], device="cuda")
    at = hq.KVAttention(a, b, 2)
    got = at.tree(q, kd, vd, m, torch.empty(n_q, 2 * heads, 128, device="cuda"))
    want = at.tree(q, *(torch.empty(heads, n_q, 128, dtype=x.dtype, device="cuda").copy_(t) for t in (kd, vd)), m,
                   torch.empty(n_q, 2 * heads, 128, device="cuda"))
    assert torch.equal(got, want)
    keep = T.seen(n_q, 40, 0, 0, m.tolist())
    kk, vv = (torch.cat((T.vectors(c), t.double()), 1) for c, t in ((a, kd), (b, vd)))
    T.check(got, None, q, kk, vv, keep, 2, 128 ** -0.5, 1)


def test_other_strides_are_still_refused():
    import lattice_entropy_coded_b200 as hq
    a, b = T.pair(2, [40], "E8")
    x = torch.randn(3, 4, 128, device="cuda").to(torch.bfloat16)
    kd, vd = torch.randn(2, 3, 128, device="cuda").to(torch.bfloat16), x[:, :2].transpose(0, 1)
    with pytest.raises(AssertionError):
        hq.KVAttention(a, b, 2).tree(x, kd, vd, torch.tensor([1, 3, 7], device="cuda"), torch.empty(3, 4, 128, device="cuda"))
