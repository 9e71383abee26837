"""The attention over the 4-bit cache where numbers are far apart: values of any
size beside one another and beside records of zeros, capped scores, scores far
below zero, and queries at the ends of their type.  Against the oracle in 64
bits, with the tolerances of test_gpu_cache.py unless a test derives its own."""
import numpy as np
import pytest
import torch

import oracle.cache as OC

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from learned_kv_chunk_b200 import fm  # noqa: E402  (loads libfm.so; raises if missing)
from tests.test_gpu_cache import DEV, TYPES, check_attention, dev, make_cache  # noqa: E402

PAGE = 16


def pages_of(x):
    """[B, heads, n, 128] fp64 -> (pages, table): the records of the values (n a multiple of a page)."""
    B, H, n, _ = x.shape
    codes, scales = OC.quant4(x)
    per = n // PAGE
    blk = np.concatenate([codes.reshape(B, H, per, PAGE * 64), scales.reshape(B, H, per, PAGE * 4)], axis=-1)
    return (np.ascontiguousarray(blk.transpose(0, 2, 1, 3)).reshape(B * per, H, PAGE * 68),
            np.arange(B * per, dtype=np.int32).reshape(B, per))


def check(q, k, v, lens, **kw):
    """q [B, Tq, Hq, 128] torch, k and v [B, heads, n, 128] fp64, held as their records."""
    kp, table = pages_of(k)
    vp, _ = pages_of(v)
    o = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.asarray(lens, np.int32)), **kw)
    check_attention(o, q, kp, vp, table, lens, PAGE, **kw)


def queries(rng, dtype, B=1, Tq=1, Hq=8, spread=1.0):
    return torch.from_numpy(spread * rng.standard_normal((B, Tq, Hq, 128))).to(TYPES[dtype])


# --------------------------------------------------- values of any size


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("Hq", [4, 12])
def test_every_token_counts_in_the_sum_whatever_its_size(dtype, Hq):
    """Two tokens of one score, 2^100 and 2^-40: each has half of the weight."""
    rng = np.random.default_rng(1)
    for big, small in ((100, -40), (125, -126), (60, -100)):
        for order in (0, 1):
            k, v = np.zeros((1, 1, 16, 128)), np.zeros((1, 1, 16, 128))
            v[0, 0, order] = 2.0 ** big * rng.choice([1.0, 3.0, 6.0], 128)
            v[0, 0, 1 - order] = 2.0 ** small
            q = queries(rng, dtype, Hq=Hq)
            check(q, k, v, [2])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("Hq,n", [(4, 3200), (12, 400), (12, 3200)])
def test_a_huge_value_leaves_the_weights_of_ordinary_ones(dtype, Hq, n):
    """One token of 6 * 2^125 some units above the others, whose weights of 2^-10 each add up to as much as its own."""
    rng = np.random.default_rng(2)
    k, v = np.zeros((1, 1, n, 128)), rng.standard_normal((1, 1, n, 128))
    for at in (0, n // 2, n - 1):
        k[0, 0] = 0.0
        k[0, 0, at, 0] = 6.0
        w = v.copy()
        w[0, 0, at] = 6.0 * 2.0 ** 125
        q = torch.zeros(1, 1, Hq, 128, dtype=TYPES[dtype])
        q[..., 0] = torch.linspace(8.0, 14.0, Hq)  # scores of 4.2 to 7.4
        check(q, k, w, [n])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_many_values_at_the_ends_of_the_scales(dtype):
    """Thousands of tokens of 2^-126 or of 6 * 2^125: neither their sum nor their weights' leaves the range."""
    rng = np.random.default_rng(3)
    for size in (2.0 ** -124, 2.0 ** -110, 2.0 ** 110, 2.0 ** 125):
        n = 9600
        k = np.zeros((1, 1, n, 128))
        v = size * rng.choice([1.0, 2.0, 6.0], (1, 1, n, 128))
        q = queries(rng, dtype)
        check(q, k, v, [n])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("Hq,Tq", [(4, 1), (12, 1), (6, 3)])
@pytest.mark.parametrize("size", [0, -15, -30, -60])
def test_records_of_zeros_among_small_values(dtype, Hq, Tq, size):
    """A value of zeros takes its weight and nothing else: the others keep their accuracy."""
    if dtype == "fp16" and size < -15:
        pytest.skip("below fp16's numbers")
    rng = np.random.default_rng(4)
    n = 320
    k = rng.standard_normal((1, 2, n, 128))
    v = 2.0 ** size * rng.standard_normal((1, 2, n, 128))
    for zeros in (np.arange(n) % 3 == 1, np.arange(n) == 5, np.arange(n) >= 7):
        w = np.where(zeros[None, None, :, None], 0.0, v)
        q = queries(rng, dtype, Tq=Tq, Hq=2 * Hq)
        check(q, k, w, [n])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_sizes_mixed_at_random(dtype):
    rng = np.random.default_rng(5)
    n = 2000
    for lo, hi in ((-120, 120), (-40, 40), (-20, 0)):
        k = rng.standard_normal((2, 2, n, 128))
        v = rng.standard_normal((2, 2, n, 128)) * np.exp2(rng.integers(lo, hi, (2, 2, n, 1)))
        v[:, :, rng.random(n) < 0.1] = 0.0
        v[:, :, 700:1200] = rng.standard_normal((2, 2, 500, 128))  # whole tiles of ordinary ones
        for Hq in (6, 24):
            q = queries(rng, dtype, B=2, Hq=Hq)
            check(q, k, v, [n, n - 3])


# -------------------------------------------------------- capped scores


@pytest.mark.parametrize("softcap", [0.5, 2.0, 20.0, 30.0, 50.0, 64.0, 300.0])
@pytest.mark.parametrize("G", [8, 16])
@pytest.mark.parametrize("general", [False, True])
def test_capped_scores_of_fp32_queries_are_those_of_fp32(softcap, G, general):
    """Two tokens, scores x and 0 (|x| <= 1), values 1 and -1: out = tanh(capped(x) / 2).

    An error dx of a logit moves out by at most dx / 2.  dx: the query's two
    pieces 2^-23 |x|, four products and constants 2^-24 |x| each, tanhf two units
    (2^-22 |x|), together below 2^-20 |x|; and the running maximum taken off and
    its base added, which are held near 8: 2^-21 in log2 units, 0.7 of that in x,
    twice for either token, below 2^-19.5.  The weights: exp2 to 2^-22 of either,
    two pieces to 2^-23 of either, a quotient: 2.5 * 2^-22.  No term has the cap."""
    rng = np.random.default_rng(6)
    B, Hkv = 8, 8
    x = rng.uniform(-1, 1, (B, Hkv * G)).astype(np.float32)
    q = torch.zeros(B, 1, Hkv * G, 128)
    q[:, 0, :, 0] = torch.from_numpy(x)
    kp, vp = (np.zeros((1, Hkv, PAGE * 68), np.uint8) for _ in range(2))
    for p in (kp, vp):
        p[:, :, PAGE * 64:] = 127
    if general:
        kp[:, :, PAGE * 64 + 3] = 0  # a group of zeros of the first key
    kp[:, :, 0] = 2               # the first key: 1 in its first dim
    vp[:, :, :64], vp[:, :, 64:128] = 0x22, 0xaa
    o = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(np.zeros((B, 1), np.int32)),
                            dev(np.full(B, 2, np.int32)), scale=1.0, softcap=softcap)
    x = x.astype(np.float64)
    want = np.tanh(softcap * np.tanh(x / softcap) / 2)[:, None, :, None]
    tol = 0.5 * (2.0 ** -20 * np.abs(x) + 2.0 ** -19.5) + 2.5 * 2.0 ** -22
    off = np.abs(o.double().cpu().numpy() - want)
    assert (off <= tol[:, None, :, None]).all(), off.max()


@pytest.mark.parametrize("softcap", [1.0, 5.0, 20.0, 50.0])
def test_caps_cost_fp32_calls_no_accuracy(softcap):
    """Scores from a few units to far past the cap, every shape of the call: the tolerance has no term of the cap."""
    rng = np.random.default_rng(7)
    lens = [300, 41, 700]
    for spread, Hq in ((0.05, 8), (0.5, 24), (3.0, 8)):
        kp, vp, table = make_cache(rng, lens, 2, PAGE)
        q = torch.from_numpy(spread * rng.standard_normal((3, 2, Hq, 128))).float()
        o = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.asarray(lens, np.int32)), softcap=softcap)
        k, there = OC.read_cache(kp, table, PAGE)
        v, _ = OC.read_cache(vp, table, PAGE)
        ref, _, abs_v, top_v = OC.attention(q.double().numpy(), k, v, there, lens, softcap=softcap)
        _, err_x, _, _ = OC.attention(q.double().numpy(), k, v, there, lens)
        tol = (2 * 2.0 ** -20 * err_x + 2.0 ** -20 + 2.0 ** -23 * (700 / 16 + 16)) * abs_v + top_v + 2.0 ** -24 * np.abs(ref) + 1e-37
        assert (np.abs(o.double().cpu().numpy() - ref) <= tol).all()


# ------------------------------------------------- scores far from zero


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("Hq,tokens", [(4, 60), (12, 60), (4, 3000), (12, 3000)])
@pytest.mark.parametrize("slope", [1e20, 2e30, 1e34])
def test_rows_whose_scores_are_all_far_below_zero(dtype, Hq, tokens, slope):
    """A kept list without the newest tokens and a steep bias: the nearest kept token has the whole weight, in
    whichever CTA or warp it is.  Its weight over itself is 1 within the f16 weights' 2^-11 (fp32: 2^-20)."""
    rng = np.random.default_rng(8)
    lens = [tokens, tokens - 1]
    kp, vp, table = make_cache(rng, lens, 1, PAGE, hi=128)
    near = [tokens // 2, 7]
    idx = np.stack([np.r_[np.arange(n), n, np.full(tokens - n - 1, -1)] for n in near])
    order = rng.permutation(tokens)
    count = np.full(2, tokens)
    q = torch.from_numpy(rng.standard_normal((2, Hq, 128))).to(TYPES[dtype])
    o = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.asarray(lens, np.int32)),
                            slopes=torch.full((Hq,), slope, device=DEV), idx=dev(idx[:, order].astype(np.int32)),
                            count=dev(count.astype(np.int32)))
    v, _ = OC.read_cache(vp, table, PAGE)
    for b in range(2):
        want = v[b, 0, near[b]]
        tol = (2.0 ** -20 if dtype == "fp32" else 2.0 ** -11 + 2.0 ** -8) * np.abs(want)
        assert (np.abs(o[b].double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("Hq", [4, 12])
@pytest.mark.parametrize("scale,softcap", [(2.0 ** 32, 2.0 ** -32), (-2.0 ** 32, 2.0 ** -32), (2.0 ** 32, 0.0), (0.1, 0.0),
                                           (1.0, 2.0 ** -32)])
@pytest.mark.parametrize("key_scale", [0, 127, 252])
def test_products_of_zero_stay_zero_whatever_multiplies_them(dtype, Hq, scale, softcap, key_scale):
    """The largest queries against keys of zeros, or keys whose only elements meet zeros of the query: every score is
    0, and the output the mean of the values."""
    rng = np.random.default_rng(9)
    n = 40
    _, vp, table = make_cache(rng, [n], 1, PAGE)
    kp = np.zeros_like(vp)
    kp[:, :, PAGE * 64:] = key_scale
    if key_scale:
        kp[:, :, :PAGE * 64:64] = 0x70  # dim 1 of every key: 6
    q = torch.zeros(1, 1, Hq, 128, dtype=TYPES[dtype])
    q[..., 0] = torch.finfo(TYPES[dtype]).max
    o = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.array([n], np.int32)), scale=scale, softcap=softcap)
    v, _ = OC.read_cache(vp, table, PAGE)
    want, size = v[0, 0, :n].mean(0), np.abs(v[0, 0, :n]).mean(0)
    tol = (2.0 ** -18 if dtype == "fp32" else 2.0 ** -11 + 2.0 ** -8) * size
    assert (np.abs(o[0, 0].double().cpu().numpy() - want) <= tol).all()


# --------------------------------------------- what the f16 operands cost


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("G", [4, 12])
@pytest.mark.parametrize("below", [8, 20, 24, 28, 32, 40])
def test_query_elements_far_below_the_largest(dtype, G, below):
    """The head's largest element meets zeros of the keys; the others are 2^-below of it and make the score.  A query
    element is off by 2^-22 of itself (fp32; 16-bit ones by nothing) and 2^-32 of the head's largest."""
    if dtype == "fp16" and below > 20:
        pytest.skip("fp16 ends there")
    rng = np.random.default_rng(below)
    n, top = 64, 8.0
    q = top * 2.0 ** -below * rng.uniform(0.5, 1, (1, 1, 2 * G, 128)) * rng.choice([-1, 1], (1, 1, 2 * G, 128))
    q[..., 0] = top
    q = torch.from_numpy(q).to(TYPES[dtype])
    k = 2.0 ** (below - 6) * rng.uniform(0.5, 6, (1, 2, n, 128)) * rng.choice([-1, 1], (1, 2, n, 128))
    k[..., 0] = 0.0
    kp, table = pages_of(k)
    vp, _ = pages_of(rng.standard_normal((1, 2, n, 128)))
    o = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.array([n], np.int32)))
    k, there = OC.read_cache(kp, table, PAGE)
    v, _ = OC.read_cache(vp, table, PAGE)
    ref, err_x, abs_v, top_v = OC.attention(q.double().numpy(), k, v, there, [n])
    narrow = dtype != "fp32"
    dx = 2.0 ** -32 * top * np.abs(k[0]).sum(-1).max() * 128 ** -0.5 + (0.0 if narrow else 2.0 ** -22) * err_x + 2.0 ** -20 * err_x
    w = (2.0 ** -11 if narrow else 2.0 ** -20) + 2.0 ** -23 * 20
    half = torch.finfo(TYPES[dtype]).eps / 2
    tol = (2 * dx + w) * abs_v + top_v + half * np.abs(ref) + 2.0 ** -25
    assert (np.abs(o.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("below", [10, 16, 22, 24, 25, 26, 40, 126])
def test_groups_far_below_their_record(dtype, below):
    """Dims 96..127 of every key and value are 2^-below of the others: off by at most 2^-25 of the record's largest
    scale where they are kept, or by themselves, at most 6 * 2^-25 of it, where they are not."""
    rng = np.random.default_rng(below)
    n, G = 64, 8
    small = np.where(np.arange(128) < 96, 1.0, 2.0 ** -below)
    q = torch.from_numpy(rng.standard_normal((1, 1, G, 128))).to(TYPES[dtype])
    x = [rng.standard_normal((1, 1, n, 128)) * small for _ in range(2)]
    x[1][..., 5, :] = 0.0  # (the tile takes the general form whatever the group's scale)
    (kp, table), (vp, _) = pages_of(x[0]), pages_of(x[1])
    o = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.array([n], np.int32)))
    k, there = OC.read_cache(kp, table, PAGE)
    v, _ = OC.read_cache(vp, table, PAGE)
    ref, err_x, abs_v, top_v = OC.attention(q.double().numpy(), k, v, there, [n])
    narrow = dtype != "fp32"
    # a largest element is at least 3 of its scale, as it was quantised: 2^-25 and 6 * 2^-25 of the scale are at most 2^-24
    # of the element
    lost = 2.0 ** -24
    dx = lost * np.abs(q.double().numpy()).sum(-1, keepdims=True) * np.abs(k).max() * 128 ** -0.5 + 2.0 ** -20 * err_x
    w = (2.0 ** -11 if narrow else 2.0 ** -20) + 2.0 ** -23 * 20
    half = torch.finfo(TYPES[dtype]).eps / 2
    tol = (2 * dx + w) * abs_v + lost * np.abs(v).max() + top_v + half * np.abs(ref)
    assert (np.abs(o.double().cpu().numpy() - ref) <= tol).all()


# ------------------------------------------------------ queries not finite


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("tokens,Hq", [(30, 4), (30, 12), (3000, 4), (3000, 12)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_query_that_is_not_finite_gives_nan_and_the_others_do_not(dtype, tokens, Hq, bad):
    """Its scores are infinite or NaN, whichever sign the keys give them; one that sees nothing gives 0 all the same."""
    rng = np.random.default_rng(10)
    kp, vp, table = make_cache(rng, [tokens, 1], 1, PAGE)
    kp[:, :, :PAGE * 64:64] = (kp[:, :, :PAGE * 64:64] & 0xf0) | 3  # dim 0 of every key: 1.5 of its scale
    q = torch.from_numpy(rng.standard_normal((2, 2, Hq, 128))).to(TYPES[dtype])
    good = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.array([tokens, 1], np.int32)))
    q[:, :, 1, 0] = bad
    o = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.array([tokens, 1], np.int32)))
    assert bool(torch.isnan(o[0, :, 1]).all()) and bool(torch.isnan(o[1, 1, 1]).all())
    assert not o[1, 0].any()  # before the row's start
    rest = [h for h in range(Hq) if h != 1]
    assert torch.equal(o[:, :, rest], good[:, :, rest])
    if bad == bad:  # a cap makes the scores cap or -cap: all the same here, and the output the mean
        o = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.array([tokens, 1], np.int32)), softcap=30.0)
        v, _ = OC.read_cache(vp, table, PAGE)
        for t in range(2):
            seen = v[0, 0, :tokens - 1 + t]
            tol = (2.0 ** -18 if dtype == "fp32" else 2.0 ** -11 + 2.0 ** -8) * np.abs(seen).mean(0) + 2.0 ** -23 * tokens / 16
            assert (np.abs(o[0, t, 1].double().cpu().numpy() - seen.mean(0)) <= tol).all()
