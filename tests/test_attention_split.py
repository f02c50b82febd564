"""How many chunks a window is taken to reach (hq_kv_attention splits its work by it): never fewer than it does, whether
tokens were appended singly behind it or dropped before it."""
import os
import random
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <stdio.h>
#include "hq_internal.h"
int main() {
    hq_kv_cache c = {};
    long long heads, tokens, chunks, window, span;
    while (scanf("%lld %lld %lld %lld %lld", &heads, &tokens, &chunks, &window, &span) == 5) {
        c.heads = (int)heads, c.tokens = tokens, c.chunks = chunks;
        const hq::ChunkCount n = hq::visible_chunks(c, window, span);
        printf("%llu %llu\n", (unsigned long long)n.most, (unsigned long long)n.likely);
    }
}
"""


def _chunks(appends):
    """[(first position, tokens)] of a head's chunks, from appends (first position, tokens)."""
    return [(t + i, min(32, n - i)) for t, n in appends for i in range(0, n, 32)]


def _reached(chunks, tokens, window, sinks, n_q):
    lo = tokens - n_q - window + 1
    return sum(1 for t, n in chunks if t + n > lo or t < sinks)


def _line_up(sizes, at=0):
    out = []
    for n in sizes:
        out.append((at, n))
        at += n
    return out


def _cases(rng):
    for _ in range(400):
        big = [rng.choice((1, 16, 31, 32, 33, 100, 256, 4096)) for _ in range(rng.randint(1, 12))]
        yield _line_up(big + [rng.choice((1, 1, 7)) for _ in range(rng.choice((0, 0, 3, 200)))])      # nothing dropped
        n = rng.choice((5, 64, 512, 4096))
        far = rng.choice((50000, 131072, 1 << 33))
        yield [(0, 4), (far, n)] + _line_up([1] * rng.choice((0, 0, 1, 100)), far + n)                # sinks and the end


def test_never_fewer_than_the_window_reaches(tmp_path):
    src, exe = tmp_path / "split.cc", tmp_path / "split"
    src.write_text(PROGRAM)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.run(["g++", "-std=c++17", f"-I{ROOT}/include", f"-I{ROOT}/lattice_entropy_coded_b200/csrc", f"-I{cuda}/include",
                    f"-L{cuda}/lib64", str(src), "-o", str(exe), "-lcudart"], check=True, capture_output=True)
    rng, lines, want = random.Random(7), [], []
    for appends in _cases(rng):
        chunks, tokens = _chunks(appends), sum(appends[-1])
        heads, n_q, sinks = rng.choice((1, 8)), rng.choice((1, 5)), rng.choice((0, 4))
        for window in (0, 1, 64, 512, 4096):
            lines.append(f"{heads} {tokens} {heads * len(chunks)} {window} {window + n_q + sinks}")
            want.append((len(chunks) if not window else _reached(chunks, tokens, window, sinks, n_q), len(chunks), window))
    run = subprocess.run([str(exe)], input="\n".join(lines), text=True, capture_output=True, check=True,
                         env={**os.environ, "LD_LIBRARY_PATH": f"{cuda}/lib64"})
    got = [tuple(map(int, x.split())) for x in run.stdout.splitlines()]
    assert len(got) == len(want)
    for line, (most, likely), (reached, there, window) in zip(lines, got, want):
        assert reached <= most <= there and 1 <= likely <= there, line
        if not window:
            assert most == likely == there, line


@pytest.mark.gpu
@pytest.mark.parametrize("heads,group,n_q", [(8, 1, 1), (2, 4, 3), (8, 4, 5)])
@pytest.mark.parametrize("ones", [0, 70])
def test_attention_over_an_evicted_cache(heads, group, n_q, ones):
    """Sinks and the last tokens of a long text, some appended singly since: against the definition in 64 bits."""
    import kvtest as T
    import lattice_entropy_coded_b200 as hq
    total, last = 20000, 1000
    pair = []
    for c in T.pair(heads, [4096] * 4 + [3616], "E8"):
        d = hq.KVCache(heads, last + 200, c.cache.params, bits_per_scalar=16.0, max_appends=100, max_append_tokens=64)
        c.repack(d, [(0, 4), (total - last, total)])
        g = torch.Generator(device="cuda").manual_seed(7)
        for _ in range(ones):
            d.append(torch.randn(heads, 1, 128, generator=g, device="cuda").to(torch.bfloat16), T.ALPHA["E8"])
        pair.append(d)
    q = torch.randn(n_q, heads * group, 128, device="cuda").to(torch.bfloat16)
    n = pair[0].tokens
    for window in (1, 100, last):
        out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda")
        hq.KVAttention(*pair, group, window=window, sinks=4)(q, out, lse=lse)
        t = torch.arange(n, device="cuda")
        pos = n - n_q + torch.arange(n_q, device="cuda")[:, None]
        keep = (t <= pos) & ((t > pos - window) | (t < 4)) & ((t < 4) | (t >= total - last))
        T.check(out, lse, q, T.vectors(pair[0]), T.vectors(pair[1]), keep, group, 128 ** -0.5, 1)
