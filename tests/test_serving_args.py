"""Refusals of the KV serving operators: every bad argument is an error before anything is enqueued (so they run
without a GPU)."""
import ctypes as C

import pytest

P = 1 << 20          # a pointer that nothing follows: a refused call reads no memory


def _hq():
    import lattice_entropy_coded_b200 as hq
    return hq


def test_struct_layouts_match_header():
    hq = _hq()
    assert C.sizeof(hq.hq_attn_spec) == 40 and hq.hq_attn_spec.scale.offset == 24 and hq.hq_attn_spec.group.offset == 32
    assert C.sizeof(hq.hq_rope_spec) == 16 and hq.hq_rope_spec.eps.offset == 12


def _cache(at, heads=2, tokens=100, chunks=8, appends=1, **kw):
    hq = _hq()
    p = dict(lattice="E8", alpha=1.0, rice_k=1, seed=at, dither=1)
    p.update(kw)
    b = P * at * 64
    return hq.hq_kv_cache(b, 4096, b + P, 64, b + 2 * P, 8, b + 3 * P, b + 4 * P, heads, 128, hq.make_params(**p), tokens,
                          chunks, appends)


def _attn(tree=False, k=None, v=None, spec=None, **kw):
    hq = _hq()
    k, v = k or _cache(1), v or _cache(2)
    sp = dict(length=100, scale=0.1, n_q=2, group=4)
    sp.update(spec or {})
    sp = hq.attn_spec(**sp)
    a = dict(q=P, qt=1024, qh=128, kd=P, vd=P, dt=128, dh=256, mask=P, out=P, dtype=0, ot=1024, oh=128, lse=None, ws=P,
             wsb=1 << 40)
    a.update(kw)
    if tree:
        return hq._lib.hq_kv_tree_attention(C.byref(k), C.byref(v), C.byref(sp), a["q"], a["qt"], a["qh"], a["kd"], a["vd"],
                                            a["dt"], a["dh"], a["mask"], a["out"], a["dtype"], a["ot"], a["oh"], a["lse"],
                                            a["ws"], a["wsb"], None)
    return hq._lib.hq_kv_attention(C.byref(k), C.byref(v), C.byref(sp), a["q"], a["qt"], a["qh"], a["out"], a["dtype"],
                                   a["ot"], a["oh"], a["lse"], a["ws"], a["wsb"], None)


BAD_ATTENTION = [
    dict(q=None), dict(q=P + 2), dict(qt=4), dict(qt=-8), dict(qh=4), dict(qh=-8), dict(out=None), dict(out=P + 8),
    dict(dtype=2), dict(ot=120), dict(oh=120), dict(oh=132), dict(ot=-1024), dict(oh=130, dtype=1), dict(lse=P + 1),
    dict(ws=None), dict(ws=P + 8), dict(wsb=64), dict(spec=dict(length=-1)), dict(spec=dict(length=101)),
    dict(spec=dict(window=-1)), dict(spec=dict(sinks=-1)), dict(spec=dict(scale=float("nan"))),
    dict(spec=dict(scale=float("inf"))), dict(spec=dict(n_q=-1)), dict(spec=dict(group=0)),
]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("bad", BAD_ATTENTION, ids=str)
def test_attention_refuses(tree, bad):
    assert _attn(tree, **bad) == _hq().HQ_EINVAL


@pytest.mark.parametrize("bad", [dict(kd=None), dict(vd=None), dict(kd=P + 8), dict(vd=P + 8), dict(dt=4), dict(dt=-8),
                                 dict(dh=-8), dict(dh=100), dict(mask=None), dict(mask=P + 4)], ids=str)
def test_tree_refuses(bad):
    assert _attn(True, **bad) == _hq().HQ_EINVAL


def test_attention_refuses_caches_that_do_not_match():
    hq = _hq()
    same = _cache(1)
    assert _attn(k=same, v=same) != hq.HQ_OK          # (byref of one object: one address)
    assert _attn(v=_cache(2, heads=3)) == hq.HQ_EINVAL
    assert _attn(v=_cache(2, chunks=9)) == hq.HQ_EINVAL
    assert _attn(v=_cache(2, appends=2)) == hq.HQ_EINVAL
    assert _attn(v=_cache(2, tokens=99)) == hq.HQ_EINVAL
    assert _attn(v=_cache(2, lattice="Z")) == hq.HQ_EUNSUPPORTED
    assert _attn(v=_cache(2, dither=0)) == hq.HQ_EUNSUPPORTED
    assert _attn(spec=dict(n_q=65)) == hq.HQ_EUNSUPPORTED
    assert _attn(spec=dict(group=65)) == hq.HQ_EUNSUPPORTED
    assert _attn(spec=dict(length=1, n_q=2)) == hq.HQ_EINVAL      # the queries are cached tokens
    assert _attn(spec=dict(n_q=0), q=None, out=None, ws=None) == hq.HQ_OK


def test_attention_workspace():
    hq = _hq()
    for heads in (1, 8, 200):
        for n_q, group in ((1, 1), (1, 4), (64, 4), (64, 64)):
            need = hq.hq_kv_attention_workspace_bytes(heads, hq.attn_spec(1000, 1.0, n_q, group))
            assert need % 256 == 0 and need >= heads * n_q * group * 520
            # one size for every length
            assert need == hq.hq_kv_attention_workspace_bytes(heads, hq.attn_spec(0, 1.0, n_q, group))
    for bad in (0, -1):
        with pytest.raises(hq.HQError, match="invalid"):
            hq.hq_kv_attention_workspace_bytes(bad, hq.attn_spec(1, 1.0, 1, 1))


def _repack(src=None, dst=None, ranges=((0, 100),), ws=P, wsb=1 << 40):
    hq = _hq()
    src, dst = src or _cache(1), dst or _cache(2, tokens=0, chunks=0, appends=0, seed=1)
    r, n = hq._ranges(ranges)
    return hq._lib.hq_kv_repack(C.byref(src), C.byref(dst), r, n, ws, wsb, None)


@pytest.mark.parametrize("ranges", [[(0, 101)], [(5, 5)], [(6, 5)], [(-1, 5)], [(0, 5), (4, 9)], [(50, 60), (0, 5)]])
def test_repack_refuses_ranges(ranges):
    assert _repack(ranges=ranges) == _hq().HQ_EINVAL


def test_repack_refuses():
    hq = _hq()
    assert _repack(ws=None) == hq.HQ_EINVAL
    assert _repack(ws=P + 4) == hq.HQ_EINVAL
    assert _repack(wsb=100) == hq.HQ_EINVAL
    assert _repack(ranges=[(2 * i, 2 * i + 1) for i in range(33)]) == hq.HQ_EUNSUPPORTED
    for other in (dict(heads=3), dict(lattice="D4"), dict(rice_k=2), dict(dither=0), dict(dk_last=1), dict(seed=9)):
        kw = dict(seed=1)
        kw.update(other)
        assert _repack(dst=_cache(2, tokens=0, chunks=0, appends=0, **kw)) == hq.HQ_EINVAL, other
    same = _cache(1)
    assert _repack(src=same, dst=_cache(1)) == hq.HQ_EINVAL        # the same buffers
    few = _cache(2, seed=1)
    few.offsets_cap = 8                                               # 8 chunks need 9 offsets
    assert _repack(dst=few) == hq.HQ_EINVAL
    few = _cache(2, seed=1)
    few.table_cap = 1
    assert _repack(dst=few, ranges=[(0, 5), (6, 7)]) == hq.HQ_EINVAL


def test_a_refused_repack_leaves_the_destination():
    dst = _cache(2, tokens=40, chunks=4, appends=3, seed=1)
    _repack(dst=dst, ranges=[(0, 101)])
    assert (dst.tokens, dst.chunks, dst.appends) == (40, 4, 3)


def _rope(spec=None, **kw):
    hq = _hq()
    s = dict(rot_dim=128, interleaved=0, norm=1, eps=1e-6)
    s.update(spec or {})
    a = dict(q=P, qt=1024, qh=128, hq=8, k=2 * P, kt=256, kh=128, hk=2, n=5, wq=P, wk=P, f=P, pos=P, qo=3 * P, qot=1024,
             qoh=128, ko=4 * P, kot=128, koh=640)
    a.update(kw)
    sp = hq.hq_rope_spec(s["rot_dim"], s["interleaved"], s["norm"], s["eps"])
    return hq._lib.hq_qk_norm_rope(a["q"], a["qt"], a["qh"], a["hq"], a["k"], a["kt"], a["kh"], a["hk"], a["n"], C.byref(sp),
                                   a["wq"], a["wk"], a["f"], a["pos"], 0, a["qo"], a["qot"], a["qoh"], a["ko"], a["kot"],
                                   a["koh"], None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(k=None), dict(q=P + 8), dict(qo=None), dict(ko=P + 8), dict(qt=12), dict(qh=-128), dict(kt=4),
    dict(qot=64), dict(qoh=64), dict(kot=64), dict(koh=12), dict(hq=-1), dict(hk=-1), dict(n=-1), dict(f=None), dict(f=P + 4),
    dict(pos=P + 4), dict(wq=P + 2), dict(wk=P + 8), dict(spec=dict(rot_dim=130)), dict(spec=dict(rot_dim=-2)),
    dict(spec=dict(rot_dim=3)), dict(spec=dict(interleaved=2)), dict(spec=dict(norm=2)), dict(spec=dict(eps=-1.0)),
    dict(spec=dict(eps=float("nan"))), dict(spec=dict(eps=float("inf")))], ids=str)
def test_norm_rope_refuses(bad):
    assert _rope(**bad) == _hq().HQ_EINVAL


def test_norm_rope_nothing_to_do():
    hq = _hq()
    assert _rope(n=0, q=None, k=None) == hq.HQ_OK
    assert _rope(hq=0, hk=0, q=None, k=None) == hq.HQ_OK
