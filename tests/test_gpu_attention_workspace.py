"""KVAttention's workspace is not given to others while a call on any stream uses it."""
import pytest
import torch

import kvtest as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", ["given", "handle", "current"])
@pytest.mark.parametrize("tree", [False, True])
def test_an_object_that_goes_while_its_call_runs_elsewhere(how, tree):
    import lattice_entropy_coded_b200 as hq
    a, b = T.pair(2, [300], "E8")
    q = torch.randn(5, 8, 128, device="cuda").to(torch.bfloat16)
    kd = torch.randn(2, 5, 128, device="cuda").to(torch.bfloat16)
    m = torch.tensor([(2 << i) - 1 for i in range(5)], device="cuda")
    call = (lambda at, o, **kw: at.tree(q, kd, kd, m, o, **kw)) if tree else (lambda at, o, **kw: at(q, o, **kw))
    want = call(hq.KVAttention(a, b, 4), torch.empty(5, 8, 128, device="cuda")).clone()
    out = torch.empty(5, 8, 128, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    at = hq.KVAttention(a, b, 4)
    where, size = at.workspace.data_ptr(), at.workspace.numel()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)          # the call waits a tenth of a second
        if how == "current":
            call(at, out)
    if how != "current":
        call(at, out, cuda_stream=side if how == "given" else side.cuda_stream)
    del at
    junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(j.data_ptr() != where for j in junk)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_on_the_default_stream_after_another():
    import lattice_entropy_coded_b200 as hq
    a, b = T.pair(2, [300], "E8")
    q = torch.randn(1, 8, 128, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        at = hq.KVAttention(a, b, 4)
        want = at(q, torch.empty(1, 8, 128, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(at(q, torch.empty(1, 8, 128, device="cuda")), want)
    assert torch.equal(at(q, torch.empty(1, 8, 128, device="cuda"), cuda_stream=0), want)
