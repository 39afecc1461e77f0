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
# norm

def exact_norm(g, m, k, least, most):
    """x of +-1 and +-7 with a mean square of 16, in rows; a weight from 2^least to 2^most; and y = x / 4
    * w, which with eps = 0 has no rounding but the last product's, in whatever order the squares add up."""
    x = np.where(np.arange(k) < 5 * k // 16, 7, 1) * g.choice([-1, 1], (m, k))
    x = g.permuted(x, axis=1).astype(np.float32)
    w = (np.exp2(g.uniform(least, most, k)) * g.choice([-1, 1], k)).astype(np.float32)
    return x, w, (x / np.float32(4)) * w


@pytest.mark.parametrize("k", [32, 64, 256, 1024, 4096, 8192, 11008, 16384, 16416, 32768])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("least,most", [(-3, 3), (-30, 0), (-141, -130), (90, 110)])
def test_rms_norm_gives_the_quantizers_codes(qmm, torch, k, aligned, least, most):
    """y is known to the bit, so codes, scales and sums are those of the quantizers on y, also where the
    scales are subnormal or a BitNet scale overflows."""
    m = 3
    x, w, y = exact_norm(rng_of(40, k, 200 + least), m, k, least, most)
    xs = up(x) if aligned else base.strided(x, 1, k + 3)
    assert torch.equal(xs, up(x))
    aq, ad, _ = qmm.rms_norm_q8_0(xs, up(w), 0.0)
    want = qmm.quantize_act_q8_0(up(y))
    assert torch.equal(aq, want[0]) and torch.equal(ad.view(torch.int16), want[1].view(torch.int16))
    got = qmm.rms_norm_bitnet(xs, up(w), 0.0)
    want = qmm.quantize_act_bitnet(up(y))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("k", [64, 2560, 4096, 11008, 20000])
@pytest.mark.parametrize("aligned", [True, False])
def test_rms_norm_of_rows_next_to_zero_and_zeros(qmm, torch, k, aligned):
    """Half of the weights are 0, so infinite BitNet scales meet zeros: the quantizer's codes again."""
    x, w, y = exact_norm(rng_of(41, k), 2, k, -140, -138)
    w[::2], y[:, ::2] = 0, 0
    xs = up(x) if aligned else base.strided(x, 1, k + 3)
    for got, want in zip(qmm.rms_norm_bitnet(xs, up(w), 0.0), qmm.quantize_act_bitnet(up(y))):
        assert torch.equal(got, want)


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


def check_elements(qmm, g, fmt, planes, heads, n, reach, q_scale):
    """One sequence over the planes' pages in a row: every element of the output against its own weighted
    mean of |v|, not the head's largest.  The weights' relative error as in attention_ref; and each
    token's product of a weight and a scale (f16: its weight alone), held as two f16 numbers, keeps 2^-36
    of `reach` in units of the largest weight (None: of the block's largest product), twice that where
    both are rounded."""
    kv_heads, ps, d = planes[0].shape[1:]
    q = (q_scale * g.standard_normal((1, heads * d))).astype(np.float32)
    table = np.arange(len(planes[0]), dtype=np.int32)[None]
    out, lse = run_attention(qmm, fmt, up(q), [up(p) for p in planes], up(table), up(np.array([n], np.int32)))
    out = out.cpu().numpy().astype(np.float64).reshape(heads, d)
    pos = np.arange(n)
    keys, values = base.cache_values(fmt, planes)
    scale = np.float64(np.float32(d ** -0.5))
    for h in range(heads):
        kk, vv = (c[pos // ps, h // (heads // kv_heads), pos % ps] for c in (keys, values))
        qh = q.reshape(heads, d)[h].astype(np.float64)
        s = kk @ qh * scale
        off = ((d / 8 + 16) * EPS32 * scale * (np.abs(kk) @ np.abs(qh)).max() +
               scale * d * 2.0 ** -22 * np.abs(qh).max() * np.abs(kk).max() + 2.0 ** -20)
        p = np.exp(s - s.max())
        if fmt == "f16":
            kept = reach * np.abs(vv).sum(0)
        else:
            where = pos // ps, h // (heads // kv_heads), pos % ps
            codes, scales = planes[2][where].astype(np.float64), planes[3][where].astype(np.float64)
            most = (p[:, None] * np.abs(scales)).max(0) if reach is None else np.full(d // 32, reach)
            kept = np.repeat(most, 32) * np.abs(codes).sum(0)
        tol = ((2 * off + 64 * EPS32) * (p @ np.abs(vv)) + 2.0 ** -35 * kept) / p.sum()
        assert (np.abs(out[h] - p @ vv / p.sum()) <= tol).all()


def scales_apart(g, kind, shape):
    """Value scales, and `reach` of check_elements."""
    u = 0.5 + g.random(shape)
    if kind == "blocks":  # of one token: six and three powers of ten apart
        return u * np.array([30, 3e-5, 0.03, 8e3])[np.arange(shape[-1]) % 4], None
    if kind == "a block of zeros":
        return u * (np.arange(shape[-1]) % 2) * 50, None
    if kind == "anything":
        return np.exp(g.uniform(np.log(1e-7), np.log(6e4), shape)), None
    if kind == "stretches":  # along the sequence: tiny, ordinary, large, small
        pages = np.arange(shape[0]) // 4 % 4
        return u * np.array([1e-6, 0.02, 3e4, 3e-4])[pages].reshape(-1, 1, 1, 1), 1.0
    if kind == "edges":
        return np.array([2.0 ** -14, 2.0 ** -10, 1.0, 0.0])[g.integers(0, 4, shape)], 1.0
    if kind == "subnormal":
        return u * 3e-6, 2.0 ** -10
    if kind == "one large token":
        s = u * 1e-3
        s[1, :, 3] = 3e4
        return s, 1.0
    raise ValueError(kind)


@pytest.mark.parametrize("kind", ["blocks", "a block of zeros", "anything", "stretches", "edges", "subnormal",
                                  "one large token"])
@pytest.mark.parametrize("heads,d", [(4, 128), (8, 64), (3, 96), (6, 192), (5, 256)])
@pytest.mark.parametrize("q_scale", [0.0, 1.0])
def test_attention_q8_0_value_scales_far_apart(qmm, kind, heads, d, q_scale):
    g = rng_of(33, d, heads)
    planes = make_cache(g, "q8_0", 40, 1, 16, d)
    scales, reach = scales_apart(g, kind, planes[3].shape)
    planes[3] = scales.astype(np.float16)
    check_elements(qmm, g, "q8_0", planes, heads, 635, reach, q_scale)


@pytest.mark.parametrize("sign", [1, -1])
def test_attention_q8_0_of_a_large_scale_without_weight(qmm, sign):
    """A token whose score is far below the others' and whose scale is 3e7 times theirs: nothing of it
    may be seen, and the others keep their digits."""
    g = rng_of(34)
    planes = make_cache(g, "q8_0", 19, 1, 16, 64)
    planes[3][:] = np.float16(1e-3)
    planes[3][5, 0, 9] = np.float16(3e4)
    planes[0][5, 0, 9], planes[1][5, 0, 9] = -127 * sign, np.float16(0.3)
    q = np.full((1, 4 * 64), sign, np.float32)
    check_attention(qmm, 34, "q8_0", 4, 1, 64, 16, [300], q=q, planes=planes,
                    table=np.arange(19, dtype=np.int32)[None])


@pytest.mark.parametrize("heads,d", [(4, 128), (8, 64), (3, 96), (5, 256)])
@pytest.mark.parametrize("q_scale", [0.0, 1.0])
def test_attention_f16_values_far_apart(qmm, heads, d, q_scale):
    g = rng_of(35, d, heads)
    planes = make_cache(g, "f16", 40, 1, 16, d)
    planes[1] = (planes[1] * np.exp(g.uniform(np.log(1e-4), np.log(1e4), d))).astype(np.float16)
    check_elements(qmm, g, "f16", planes, heads, 635, 1.0, q_scale)


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


# ---------------------------------------------------------------------------
# outputs

def test_large_outputs_have_memory_of_their_own(qmm, torch):
    """Keeping one output of a large call keeps only that one's bytes; small calls' outputs share 256 KB at
    most.  Contents are right in either form."""
    def owned(t):
        return t.untyped_storage().nbytes()

    def z(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    for m in (1, 16, 64, 2048):
        x, w = torch.ones((m, 4096), device="cuda"), torch.ones(4096, device="cuda")
        calls = [qmm.rms_norm_q8_0(x, w, residual=x), qmm.rms_norm_bitnet(x, w, residual=x),
                 qmm.rms_norm_bitnet(x, w)[:3],
                 qmm.log_probs(x, z(m, 8, dtype=torch.int32), top_k=32)]
        cache, table = z(4, 2, 16, 128, dtype=torch.float16), z(m, 1, dtype=torch.int32)
        calls.append(qmm.paged_attention_f16(z(m, 16 * 128), cache, cache, table, z(m, dtype=torch.int32) + 5))
        for outputs in calls:
            size = sum(t.numel() * t.element_size() for t in outputs)
            for t in outputs:
                assert owned(t) <= max(t.numel() * t.element_size(), min(1 << 18, size + 64 * len(outputs)))
            if size > 1 << 18:
                assert len({t.untyped_storage().data_ptr() for t in outputs}) == len(outputs)
        assert torch.equal(calls[0][2], x + x) and (calls[0][0] == 127).all()
        assert torch.equal(calls[1][2], calls[1][0].int().sum(-1, dtype=torch.int32))
        assert (calls[3][2] == torch.arange(32, device="cuda")).all() and (calls[4][0] == 0).all()


# ---------------------------------------------------------------------------
# errors

CHECK_TWICE = """
import time
import torch
import quantized_matmul_gb300 as q

def check():
    times = []
    for _ in range(300):
        t = time.perf_counter()
        assert q.check_device_error() == 0
        times.append(time.perf_counter() - t)
    return sorted(times)[len(times) // 2]

torch.zeros(1, device="cuda")
check()
before = check()
lens, table = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([500], [list(range(32))]))
f16 = torch.ones(32, 1, 16, 128, dtype=torch.float16, device="cuda")
codes, scales = f16.to(torch.int8), torch.ones(32, 1, 16, 4, dtype=torch.float16, device="cuda")
x = torch.ones(1, 128, device="cuda")
q.paged_attention_f16(x, f16, f16, table, lens)
q.paged_attention_q8_0(x, codes, scales, codes, scales, table, lens)
q.log_probs(torch.zeros(1, 20000, device="cuda"))
print(before / check())
"""


def test_the_error_check_reads_no_words_of_kernels_that_never_ran():
    """Five words before the first exchange within a cluster, eight after: a process that only runs the
    products pays for those (read apart, each takes about as long)."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHECK_TWICE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert float(r.stdout) < 0.85, r.stdout
