"""A repacked cache holds the dense rotation that it shares with its source, so the source may go."""
import gc

import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


def _hq():
    import lattice_entropy_coded_b200 as hq
    return hq


def _source(x):
    hq = _hq()
    src = hq.KVCache(2, 60, hq.make_params("E8", 1.0, 1, 5, 1), bits_per_scalar=16.0, max_appends=4, max_append_tokens=64,
                     rotation=hq.hq_haar_rotation(11))
    src.append(x, 0.7)
    return src


def _copy(src):
    hq = _hq()
    return src.repack(hq.KVCache(2, 100, src.cache.params, bits_per_scalar=16.0, max_appends=4, max_append_tokens=64))


def test_the_source_and_its_rotation_may_go():
    x = synth.kv(2, 60, seed=2)[0].cuda()
    more = synth.kv(2, 9, seed=3)[0].cuda()
    src = _source(x)
    want = src.read(torch.empty(2, 60, 128, device="cuda")).clone()
    whole = _copy(src)
    whole.append(more, 0.7)
    want_more = whole.read(torch.empty(2, 69, 128, device="cuda")).clone()
    dst, again = _copy(src), _copy(_copy(src))       # one of them through a cache that is gone at once
    assert dst.rotation is src.rotation and again.rotation is src.rotation
    torch.cuda.synchronize()
    del src, whole
    gc.collect()
    junk = [torch.full((128, 128), 3.0, device="cuda") for _ in range(200)]   # noqa: F841 (over what was freed)
    for d in (dst, again):
        assert torch.equal(d.read(torch.empty(2, 60, 128, device="cuda")), want)
        d.append(more, 0.7)
        assert torch.equal(d.read(torch.empty(2, 69, 128, device="cuda")), want_more)


def test_a_refused_repack_leaves_the_destination_its_rotation():
    hq = _hq()
    src = _source(synth.kv(2, 60, seed=2)[0].cuda())
    other = hq.KVCache(2, 60, hq.make_params("E8", 1.0, 1, 5, 1), max_appends=4, rotation=hq.hq_haar_rotation(12))
    mine = other.rotation
    with pytest.raises(hq.HQError):
        src.repack(other)
    assert other.rotation is mine
