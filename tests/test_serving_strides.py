"""Output strides of the KV serving operators: layouts whose vectors share an element are refused, no other is."""
import itertools
import os
import subprocess

import pytest
import torch

import test_serving_args as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRIDES = [0, 64, 120, 128, 136, 192, 256, 264, 384, 392, 512, 640, 648, 1024, 1152, (1 << 63) - 8]
COUNTS = [(1, 1), (1, 4), (2, 1), (2, 2), (3, 4), (7, 2), (2, 12), (5, 8), (64, 256), (8191, 40), (1 << 31, 65536)]

PROGRAM = r"""
#include <stdio.h>
#include "hq_internal.h"
int main() {
    long long a, b, c, d;
    while (scanf("%lld %lld %lld %lld", &a, &b, &c, &d) == 4) printf("%d\n", (int)hq::vectors_apart(a, b, c, d));
}
"""


def _shared(n0, ld0, n1, ld1):
    at = sorted(i * ld0 + j * ld1 for i in range(n0) for j in range(n1))
    return any(b - a < 128 for a, b in zip(at, at[1:]))


def test_the_rule_against_every_pair_of_vectors(tmp_path):
    src, exe = tmp_path / "apart.cc", tmp_path / "apart"
    src.write_text(PROGRAM)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.run(["g++", "-std=c++17", f"-I{ROOT}/include", f"-I{ROOT}/lattice_entropy_coded_b200/csrc", f"-I{cuda}/include",
                    f"-L{cuda}/lib64", str(src), "-o", str(exe), "-lcudart"], check=True, capture_output=True)
    cases = [(n, a, h, b) for n, h in COUNTS for a, b in itertools.product(STRIDES, STRIDES)]
    run = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, c)) for c in cases), text=True, capture_output=True,
                         check=True, env={**os.environ, "LD_LIBRARY_PATH": f"{cuda}/lib64"})
    got = [bool(int(x)) for x in run.stdout.split()]
    assert len(got) == len(cases)
    for c, ok in zip(cases, got):
        if c[0] * c[2] <= 20000:      # larger ones: that the rule answers at once
            assert ok == (not _shared(*c)), c


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("ot,oh", [(128, 128), (256, 128), (128, 136), (392, 256), (1016, 128), (136, 128)])
def test_attention_refuses_rows_that_overlap(tree, ot, oh):
    """2 queries of 8 heads."""
    assert _shared(2, ot, 8, oh)
    assert A._attn(tree, ot=ot, oh=oh) == A._hq().HQ_EINVAL
    assert A._attn(tree, ot=ot, oh=oh, dtype=1) == A._hq().HQ_EINVAL


@pytest.mark.parametrize("side", ["q", "k"])
@pytest.mark.parametrize("t,h", [(128, 128), (256, 128), (128, 256), (392, 256), (136, 128)])
def test_norm_rope_refuses_vectors_that_overlap(side, t, h):
    """5 tokens of 8 query and 3 key heads."""
    assert _shared(5, t, 8 if side == "q" else 3, h)
    bad = dict(qot=t, qoh=h) if side == "q" else dict(kot=t, koh=h, hk=3)
    assert A._rope(**bad) == A._hq().HQ_EINVAL


@pytest.mark.parametrize("bad", [dict(qo=A.P, qot=2048), dict(qo=A.P, qot=128, qoh=1024), dict(ko=2 * A.P),
                                 dict(ko=2 * A.P, kot=256, koh=1280)], ids=str)
def test_norm_rope_refuses_to_work_in_place_under_other_strides(bad):
    """The inputs lie at strides (1024, 128) and (256, 128)."""
    assert A._rope(**bad) == A._hq().HQ_EINVAL


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,heads", [(1, 4), (5, 1)])
def test_norm_rope_in_place_where_a_stride_says_nothing(tokens, heads):
    hq = A._hq()
    x = torch.randn(tokens, heads, 128, device="cuda").to(torch.bfloat16)
    f = 10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
    want = torch.empty_like(x)
    hq.hq_qk_norm_rope(x, None, hq.rope_spec(), f, want, None)
    other = x.as_strided(x.shape, (x.stride(0), 1024, 1) if heads == 1 else (4096, 128, 1))
    hq.hq_qk_norm_rope(x, None, hq.rope_spec(), f, other, None)
    assert torch.equal(x, want)


@pytest.mark.gpu
def test_vectors_that_lie_between_one_another():
    """Strides 640 and 256: the second token's vectors lie between the first's, none on another."""
    hq = A._hq()
    x = torch.randn(2, 4, 128, device="cuda").to(torch.bfloat16)
    f = 10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
    want, buf = torch.empty_like(x), torch.full((2048,), 7.0, dtype=torch.bfloat16, device="cuda")
    hq.hq_qk_norm_rope(x, None, hq.rope_spec(), f, want, None)
    out = buf.as_strided((2, 4, 128), (640, 256, 1))
    hq.hq_qk_norm_rope(x, None, hq.rope_spec(), f, out, None)
    assert torch.equal(out, want) and int((buf == 7).sum()) >= 2048 - 1024


@pytest.mark.gpu
def test_attention_rows_that_lie_between_one_another():
    import kvtest as T
    hq = A._hq()
    a, b = T.pair(2, [70], "E8")
    q = torch.randn(2, 4, 128, device="cuda").to(torch.bfloat16)
    at = hq.KVAttention(a, b, 2)
    want, buf = at(q, torch.empty(2, 4, 128, device="cuda")), torch.full((2048,), 7.0, device="cuda")
    out = buf.as_strided((2, 4, 128), (640, 256, 1))
    at(q, out)
    assert torch.equal(out, want) and int((buf == 7).sum()) == 2048 - 1024
