"""hq_qk_norm_rope against the formula in 64 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _hq():
    import lattice_entropy_coded_b200 as hq
    return hq


def _ref(x, w, pos, freq, rot, inter, norm, eps):
    """x [tokens, heads, 128] -> (y, the size of what each element is made of)."""
    x = x.double()
    if norm:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
        if w is not None:
            x = x * w.double()
    i = torch.arange(rot // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    f = pos.double()[:, None, None] * freq[: rot // 2]
    y, size = x.clone(), x.abs()
    y[..., a] = x[..., a] * f.cos() - x[..., b] * f.sin()
    y[..., b] = x[..., b] * f.cos() + x[..., a] * f.sin()
    both = x[..., a].abs() + x[..., b].abs()
    size[..., a] = both
    size[..., b] = both
    return y, size


def _check(got, x, w, pos, freq, rot, inter, norm, eps=1e-6):
    """bf16 rounds by half a step, 2^-8; before it fp32: the sum of squares (128 terms: 2^-24 64 on average of the
    half that the root leaves, at most 2^-18), the root and two products (2^-22), the sines (2^-22, their angle within
    2^-24 of a half turn), two products and a sum (2^-23): 2^-17 of the pair's size covers them."""
    y, size = _ref(x, w, pos, freq, rot, inter, norm, eps)
    err = (got.double() - y).abs()
    lim = 2.0 ** -8 * y.abs() + 2.0 ** -17 * size + 1e-38
    assert bool((err <= lim).all()), f"worst error / bound {float((err / lim).max()):.3f}"


def _freq(rot):
    return 500000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / max(rot // 2, 1))


def _case(tokens, hq_, hk, rot=128, inter=0, norm=1, weights=True, pos0=0, positions=None, seed=0, std=1.0):
    hq = _hq()
    g = torch.Generator(device="cuda").manual_seed(seed + tokens)
    qkv = (torch.randn(tokens, hq_ + 2 * hk, 128, generator=g, device="cuda") * std).to(torch.bfloat16)
    w = [(1 + 0.2 * torch.randn(128, generator=g, device="cuda")).to(torch.bfloat16) if weights else None for _ in "qk"]
    q, k = qkv[:, :hq_], qkv[:, hq_:hq_ + hk].transpose(0, 1)
    qo = torch.full((tokens, hq_, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ko = torch.full((hk, tokens, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    before = qkv.clone()
    hq.hq_qk_norm_rope(q, k, hq.rope_spec(rot, inter, norm), _freq(rot), qo, ko, w[0], w[1], positions, pos0)
    pos = positions if positions is not None else pos0 + torch.arange(tokens, device="cuda")
    _check(qo, q, w[0], pos, _freq(rot), rot, inter, norm)
    _check(ko.transpose(0, 1), k.transpose(0, 1), w[1], pos, _freq(rot), rot, inter, norm)
    assert torch.equal(qkv, before)


@pytest.mark.parametrize("rot", [0, 2, 6, 8, 10, 64, 96, 120, 126, 128])
@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("norm", [0, 1])
def test_rotations(rot, inter, norm):
    _case(5, 3, 2, rot, inter, norm, pos0=1000)


@pytest.mark.parametrize("tokens,heads_q,heads_k", [(1, 1, 1), (1, 32, 8), (2, 7, 1), (17, 24, 5), (61, 32, 8),
                                                    (1000, 9, 3), (8191, 4, 2), (33, 0, 2), (33, 3, 0)])
def test_sizes(tokens, heads_q, heads_k):
    hq = _hq()
    if heads_q and heads_k:
        return _case(tokens, heads_q, heads_k)
    x = torch.randn(tokens, heads_q + heads_k, 128, device="cuda").to(torch.bfloat16)
    o = torch.empty_like(x)
    pos = torch.arange(tokens, device="cuda")
    if heads_q:
        hq.hq_qk_norm_rope(x, None, hq.rope_spec(), _freq(128), o, None)
    else:
        hq.hq_qk_norm_rope(None, x.transpose(0, 1), hq.rope_spec(), _freq(128), None, o.transpose(0, 1))
    _check(o, x, None, pos, _freq(128), 128, 0, 1)


def test_nothing_to_do():
    hq = _hq()
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    assert hq.hq_qk_norm_rope(e, None, hq.rope_spec(), _freq(128), e, None) == hq.HQ_OK


@pytest.mark.parametrize("pos0", [0, 123457, 10 ** 7, 2 ** 40])
def test_far_positions(pos0):
    """The angle's fraction of a turn is found in 64 bits: 2^40 radians hold it to 2^-12, so does the reference."""
    if pos0 < 2 ** 30:
        return _case(9, 2, 1, pos0=pos0)
    hq = _hq()
    x = torch.randn(3, 2, 128, device="cuda").to(torch.bfloat16)
    o = torch.empty_like(x)
    freq = 2 * math.pi * 2.0 ** -torch.arange(1, 65, dtype=torch.float64, device="cuda").clamp(max=8)
    hq.hq_qk_norm_rope(x, None, hq.rope_spec(), freq, o, None, pos0=pos0)
    pos = torch.arange(3, device="cuda")         # 2^40 positions are whole turns of every frequency
    # freq is 2 pi / 2^n rounded: 2^40 positions turn by up to 2^40 2^-52 radians more
    y, size = _ref(x, None, pos, freq, 128, 0, 1, 1e-6)
    assert bool(((o.double() - y).abs() <= 2.0 ** -8 * y.abs() + 2.0 ** -9 * size).all())


def test_given_positions():
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.randint(0, 100000, (50,), generator=g, device="cuda")
    pos[7] = pos[8]
    _case(50, 8, 2, positions=pos)
    _case(50, 8, 2, positions=-pos)


@pytest.mark.parametrize("std", [1e-18, 1e-4, 1e4, 1e15])
def test_magnitudes(std):
    """Small vectors lean on eps, large ones keep their sum of squares finite."""
    _case(6, 2, 2, std=std)
    _case(6, 2, 2, std=std, norm=0, weights=False)


def test_a_vector_of_zeros_or_nan_stays_alone():
    hq = _hq()
    x = torch.randn(3, 2, 128, device="cuda").to(torch.bfloat16)
    o, o2 = torch.empty_like(x), torch.empty_like(x)
    hq.hq_qk_norm_rope(x, None, hq.rope_spec(), _freq(128), o, None)
    x[1, 0], x[2, 1, 3] = 0, float("nan")
    hq.hq_qk_norm_rope(x, None, hq.rope_spec(), _freq(128), o2, None)
    assert bool((o2[1, 0] == 0).all()) and bool(torch.isnan(o2[2, 1]).all())
    same = torch.ones(3, 2, dtype=torch.bool, device="cuda")
    same[1, 0] = same[2, 1] = False
    assert torch.equal(o[same], o2[same])


@pytest.mark.parametrize("rot,inter", [(128, 0), (64, 1), (10, 0), (128, 1)])
def test_in_place(rot, inter):
    hq = _hq()
    x = torch.randn(40, 6, 128, device="cuda").to(torch.bfloat16)
    w = torch.rand(128, device="cuda").to(torch.bfloat16)
    q, k = x[:, :4], x[:, 4:].transpose(0, 1)
    qo, ko = torch.empty(40, 4, 128, dtype=x.dtype, device="cuda"), torch.empty(2, 40, 128, dtype=x.dtype, device="cuda")
    spec = hq.rope_spec(rot, inter)
    hq.hq_qk_norm_rope(q, k, spec, _freq(rot), qo, ko, w, w)
    hq.hq_qk_norm_rope(q, k, spec, _freq(rot), q, k, w, w)
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_strided_output_leaves_the_rest():
    hq = _hq()
    x = torch.randn(9, 4, 128, device="cuda").to(torch.bfloat16)
    buf = torch.full((9, 4, 160), 3.0, dtype=torch.bfloat16, device="cuda")
    hq.hq_qk_norm_rope(x, None, hq.rope_spec(), _freq(128), buf[..., 16:144], None)
    _check(buf[..., 16:144], x, None, torch.arange(9, device="cuda"), _freq(128), 128, 0, 1)
    assert bool((buf[..., :16] == 3).all()) and bool((buf[..., 144:] == 3).all())


def test_captured_and_on_another_stream():
    hq = _hq()
    x = torch.randn(20, 4, 128, device="cuda").to(torch.bfloat16)
    pos = torch.arange(20, device="cuda")
    o, want = torch.empty_like(x), torch.empty_like(x)
    f, spec = _freq(128), hq.rope_spec()
    g = torch.cuda.CUDAGraph()
    hq.hq_qk_norm_rope(x, None, spec, f, o, None, positions=pos)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        hq.hq_qk_norm_rope(x, None, spec, f, o, None, positions=pos)
    pos += 100          # the positions are read when the graph runs
    hq.hq_qk_norm_rope(x, None, spec, f, want, None, positions=pos)
    g.replay()
    assert torch.equal(o, want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o.zero_()
    torch.cuda.synchronize()
    hq.hq_qk_norm_rope(x, None, spec, f, o, None, positions=pos, cuda_stream=side)
    side.synchronize()
    assert torch.equal(o, want)
