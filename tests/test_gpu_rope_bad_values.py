"""hq_qk_norm_rope with infinities and NaN: a pair that does not turn keeps to itself."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _run(x, rot, inter, norm):
    import lattice_entropy_coded_b200 as hq
    freq = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / max(rot // 2, 1))
    o = torch.empty_like(x)
    hq.hq_qk_norm_rope(x, None, hq.rope_spec(rot, inter, norm), freq, o, None, pos0=77)
    return o


@pytest.mark.parametrize("rot", [0, 2, 10, 64, 96, 120, 126])   # element by element, and in runs of four or eight
@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_without_norm_what_does_not_turn_passes_unchanged(rot, inter, bad):
    g = torch.Generator(device="cuda").manual_seed(rot)
    x = torch.randn(128, 3, 128, generator=g, device="cuda").to(torch.bfloat16)
    clean = _run(x, rot, inter, 0)
    assert torch.equal(clean[..., rot:], x[..., rot:])
    # a bad value in each coordinate of the rest, one token each
    at = torch.arange(rot, 128, device="cuda")
    y = x.clone()
    y[at, 1, at] = bad
    want = clean.clone()
    want[at, 1, at] = bad
    got = _run(y, rot, inter, 0)
    assert torch.equal(got.nan_to_num(12345.0, 54321.0, -54321.0), want.nan_to_num(12345.0, 54321.0, -54321.0))


@pytest.mark.parametrize("rot", [0, 10, 64])
@pytest.mark.parametrize("inter", [0, 1])
def test_with_norm_an_infinity_is_nan_and_the_rest_zero(rot, inter):
    """x / sqrt(infinity): 0 for what is finite, infinity / infinity for the rest; nothing spreads past a pair."""
    x = torch.randn(4, 2, 128, device="cuda").to(torch.bfloat16)
    x[2, 1, 101] = float("inf")
    got = _run(x, rot, inter, 1)
    assert bool(torch.isnan(got[2, 1, 101]))
    got[2, 1, 101] = 0
    assert bool((got[2, 1] == 0).all()) and bool(torch.isfinite(got).all())


def test_a_pair_that_turns_spreads_as_the_formula_does():
    x = torch.randn(2, 1, 128, device="cuda").to(torch.bfloat16)
    clean = _run(x, 64, 0, 0)
    x[1, 0, 5] = float("inf")
    got = _run(x, 64, 0, 0)
    assert not bool(torch.isfinite(got[1, 0, 5])) and not bool(torch.isfinite(got[1, 0, 37]))
    got[1, 0, 5], got[1, 0, 37] = clean[1, 0, 5], clean[1, 0, 37]
    assert torch.equal(got, clean)
