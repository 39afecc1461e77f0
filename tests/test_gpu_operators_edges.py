"""Edges of the operators around the products, against plain implementations
in 64 bits, beside those of test_gpu_operators.py, whose helpers and derived
tolerances they share."""
import numpy as np
import pytest

import test_gpu_operators as base
from test_gpu_operators import EPS32, check_attention, check_log_probs, make_cache, rng_of, run_attention, up

pytestmark = pytest.mark.gpu


@pytest.fixture
def torch():
    return pytest.importorskip("torch")


# ---------------------------------------------------------------------------
# attention

@pytest.mark.parametrize("fmt", ["f16", "q8_0"])
@pytest.mark.parametrize("scale", [0.02, 1e-4])
@pytest.mark.parametrize("first", [31488, 65536 + 31488])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 160, 192, 224, 256])
def test_attention_does_not_depend_on_where_the_pages_lie(qmm, torch, fmt, d, first, scale):
    """The same tokens in the cache's first pages and in pages from row `first` on, whose number's bits
    would be a large f16: the same bits out.  For one sequence and a ragged batch."""
    g = rng_of(31, d)
    kv_heads, ps, used = 2, 16, 38
    planes = make_cache(g, fmt, used, kv_heads, ps, d)
    if fmt == "q8_0":
        planes[3] = (scale * (0.5 + g.random(planes[3].shape))).astype(np.float16)
    at = first // (kv_heads * ps)
    low, high = [up(p) for p in planes], []
    for p in low:
        high.append(torch.zeros((at + used,) + p.shape[1:], dtype=p.dtype, device="cuda"))
        high[-1][at:] = p
    for lens in ([300], [40, 300]):
        table = g.permutation(used).astype(np.int32)[: 19 * len(lens)].reshape(len(lens), 19)
        q = up(g.standard_normal((len(lens), 6 * d), np.float32))
        n = up(np.array(lens, np.int32))
        want = run_attention(qmm, fmt, q, low, up(table), n)
        got = run_attention(qmm, fmt, q, high, up(table + at), n)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("fmt", ["f16", "q8_0"])
@pytest.mark.parametrize("d,kv_heads,n", [(32, 640, 32768), (128, 640, 8192), (256, 320, 8200)])
def test_attention_of_long_sequences_without_splits(qmm, torch, fmt, d, kv_heads, n):
    """A zero query and values above zero: the output is their mean, whose sum runs through n / 64 (n /
    128 for d <= 64) tiles a warp.  Additions rounded to nearest are off by 2^-24 / sqrt(3) of a partial
    sum each and independent, 2^-24 sqrt(tiles) / 3 in all; six times that, and four roundings (halves,
    joins, the quotient), bound every element.  Their mean over all elements is a bias: the sums of one
    tile (of at most 2^-23 for the order of 16 products and of its two halves) and the roundings after."""
    page = 64
    pages = -(-n // page)
    gen = torch.Generator(device="cuda").manual_seed(d)
    shape = (pages, kv_heads, page, d)
    if fmt == "f16":
        v = torch.rand(shape, generator=gen, device="cuda", dtype=torch.float16)
        planes, values = [v, v], v
    else:
        codes = torch.randint(0, 128, shape, generator=gen, device="cuda", dtype=torch.int8)
        scales = torch.full(shape[:3] + (d // 32,), 0.0123, device="cuda", dtype=torch.float16)
        planes, values = [codes, scales, codes, scales], codes
    table = torch.arange(pages, device="cuda", dtype=torch.int32)[None]
    lens = torch.tensor([n], device="cuda", dtype=torch.int32)
    q = torch.zeros(1, kv_heads * d, device="cuda")
    out, lse = run_attention(qmm, fmt, q, planes, table, lens)
    total = torch.zeros(kv_heads, d, dtype=torch.float64, device="cuda")
    for p in range(pages):
        total += values[p, :, : min(page, n - p * page)].double().sum(1)
    want = total / n * (float(np.float16(0.0123)) if fmt == "q8_0" else 1.0)
    off = (out.view(kv_heads, d).double() - want) / want
    tiles = n / (128 if d <= 64 else 64)
    assert float(off.abs().max()) <= (6 * tiles ** 0.5 / 3 + 4) * EPS32
    assert abs(float(off.mean())) <= 8 * EPS32
    assert float((lse.double() - np.log(n)).abs().max()) <= (6 * tiles ** 0.5 / 3 + 16) * EPS32


@pytest.mark.parametrize("d", [160, 192, 224])
def test_attention_q8_0_in_pages_of_large_row_numbers(qmm, d):
    g = rng_of(32, d)
    check_attention(qmm, 32, "q8_0", 4, 2, d, 16, [300, 150],
                    table=(984 + g.permutation(38)).astype(np.int32).reshape(2, 19),
                    planes=make_cache(g, "q8_0", 984 + 38, 2, 16, d))


@pytest.mark.parametrize("fmt", ["f16", "q8_0"])
@pytest.mark.parametrize("heads", [1, 5, 8, 11])
def test_attention_with_heads_of_192_within_a_cluster(qmm, fmt, heads):
    for n in (129, 577, 897, 1024):
        check_attention(qmm, n, fmt, heads, 1, 192, 16, [n])


@pytest.mark.parametrize("fmt", ["f16", "q8_0"])
@pytest.mark.parametrize("garbage", [np.nan, -np.inf, 65504.0])
@pytest.mark.parametrize("d", [32, 160, 192, 224, 256])
def test_attention_of_other_head_sizes_ignores_what_it_does_not_attend_to(qmm, torch, fmt, garbage, d):
    base.test_attention_ignores_what_it_does_not_attend_to(qmm, torch, fmt, garbage, d)


# ---------------------------------------------------------------------------
# log probabilities

@pytest.mark.parametrize("m,n", [(1, 128256), (2, 40001), (16, 32768)])
@pytest.mark.parametrize("low", [0, 5])
def test_log_probs_join_of_many_alternatives(qmm, torch, m, n, low):
    """Eight CTAs a row, one of whose parts holds small words alone: the bound of the join is low, so
    nearly all of the eight times 32 alternatives are ranked.  Every repetition gives the same words."""
    g = rng_of(30, m, n, low)
    x = g.standard_normal((m, n)).astype(np.float32)
    part = n // 8
    x[:, low * part + 64: (low + 1) * part - 64] -= 30
    check_log_probs(qmm, x, 32)
    view = up(x)
    want = qmm.log_probs(view, top_k=32)
    for _ in range(200):
        got = qmm.log_probs(view, top_k=32)
        assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
