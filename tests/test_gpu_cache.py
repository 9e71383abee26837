"""The operators around the 4-bit paged cache on the GPU against the oracle in
64 bits: the append (codes, scales and values exactly), the attention (heads,
types, lengths, masks, lists, missing pages, strides), the indexer keys'
records, the residual RMSNorm, and a run of them together with the retriever.

Tolerances.  Stored codes are equal, bit for bit.  An attention output is off
by at most
    (2 dx + w) * sum p|v| + small + eps/2 * |o|
with dx the error of a logit: 2^-20 of what its terms and its cap and bias add
up to (fp32 products summed in fp32, queries split to 2^-22, exp2 and tanh to a
few 2^-23 each), w the weights' rounding (2^-11 for 16-bit types, 2^-20 for
fp32, and 2^-23 for each sixteen tokens summed), eps the output type's step.

`small` is what the f16 operands' subnormals cost.  Weights are held times 2^8
relative to the largest p * (size of v), where a record's size is its largest
scale; the steps of f16 end at 2^-24, so a weight is off by up to 2^-25 * 2^-8 =
2^-33 of the largest, and each of n tokens adds that times its largest code, 6
(6 sizes are at most 12 times the record's largest |v|: some code of the
largest group is at least 1/2).  A value far below its record's size is off by
2^-25 sizes, at most 2^-24 times the record's largest |v|, weighted by p; a key
element likewise, which adds |q| times 2^-24 max|k| to a logit (in dx, as
2^-20 / 16)."""
import math

import numpy as np
import pytest
import torch

import oracle.cache as OC
import oracle.retriever as O
from tests import helpers as H

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from learned_kv_chunk_b200 import fm  # noqa: E402  (loads libfm.so; raises if missing)

DEV = torch.device("cuda", 0)
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def make_cache(rng, lens, Hkv, page, spare=2, lo=120, hi=131, cap=None):
    """Random records: (k_pages, v_pages, table) on the host."""
    B = len(lens)
    cap = max(1, max(lens)) if cap is None else cap
    per = -(-cap // page)
    n_pages = B * per + spare

    def pool():
        p = rng.integers(0, 256, (n_pages, Hkv, page * 68), dtype=np.uint8)
        p[:, :, page * 64:] = rng.integers(lo, hi, (n_pages, Hkv, page * 4), dtype=np.uint8)
        return p

    table = rng.permutation(n_pages)[:B * per].reshape(B, per).astype(np.int32)
    return pool(), pool(), table


def check_attention(o, q, kp, vp, table, lens, page, **kw):
    k, there = OC.read_cache(kp, table, page)
    v, _ = OC.read_cache(vp, table, page)
    Tq = q.shape[1]
    with np.errstate(all="ignore"):
        ref, err_x, abs_v, top_v = OC.attention(q.double().numpy(), k, v, there, lens, **kw)
    narrow = o.dtype != torch.float32
    n = max(1, k.shape[2])
    w = (2.0 ** -11 if narrow else 2.0 ** -20) + 2.0 ** -23 * (n / 16 + 16)
    # below the type's smallest normal number (2^-14 in fp16) its steps are tiny * eps apart, whatever the value
    sub = torch.finfo(o.dtype).tiny * half_step(o.dtype) + 1e-37
    tol = (2 * 2.0 ** -20 * err_x + w) * abs_v + top_v + half_step(o.dtype) * np.abs(ref) + sub
    got = o.double().cpu().numpy().reshape(ref.shape)
    bad = np.abs(got - ref) > tol
    assert np.isfinite(got).all() and not bad.any(), (
        Tq, np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4], (np.abs(got - ref) / tol).max())


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def run_attention(rng, lens, Hq, Hkv, Tq=1, page=16, dtype="bf16", idx=None, count=None, kv_start=None, slopes=None,
                  cache=None, q_scale=1.5, **kw):
    kp, vp, table = cache if cache is not None else make_cache(rng, lens, Hkv, page)
    q = torch.from_numpy(q_scale * rng.standard_normal((len(lens), Tq, Hq, 128))).to(TYPES[dtype])
    arrays = {}
    for name, a, t in (("idx", idx, np.int32), ("count", count, np.int32), ("kv_start", kv_start, np.int32),
                       ("slopes", slopes, np.float32)):
        if a is not None:
            arrays[name] = dev(np.asarray(a, t))
    o = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.asarray(lens, np.int32)), **arrays, **kw)
    torch.cuda.synchronize()
    kw.pop("max_len", None)
    check_attention(o, q, kp, vp, table, lens, page, idx=None if idx is None else np.asarray(idx),
                    count=count, kv_start=kv_start, slopes=slopes, **kw)
    return o


# ------------------------------------------------------------------ the append


def append_case(rng, dtype, T, Hq, Hkv, page, rope_dim, B=3, first=None, positions=None, x=None):
    kind = TYPES[dtype]
    x = rng.standard_normal((T, Hq + 2 * Hkv, 128)) if x is None else x
    qkv = torch.from_numpy(x).to(kind)
    seq = np.sort(rng.integers(0, B, T)).astype(np.int32)
    first = rng.integers(0, 40, B) if first is None else first
    pos = np.zeros(T, np.int64)
    for b in range(B):
        m = seq == b
        pos[m] = first[b] + np.arange(m.sum())
    order = rng.permutation(T)  # tokens of the rows in no order
    seq, pos = seq[order], pos[order]
    pad = rng.random(T) < 0.15
    seq[pad] = rng.choice([-1, B, 1 << 30], pad.sum())
    per = int(pos.max()) // page + 1
    table = rng.permutation(B * per + 2)[:B * per].reshape(B, per).astype(np.int32)
    return qkv, seq, pos, table


def check_append(qkv, seq, pos, table, Hq, Hkv, page, rope_dim, positions=None, q_in_place=False):
    T = qkv.shape[0]
    n_pages = int(table.max()) + 3
    g = qkv.to(DEV)
    start = np.random.default_rng(9).integers(0, 256, (n_pages, Hkv, page * 68), dtype=np.uint8)
    kp, vp = dev(start), dev(start)
    freq = O.yarn_inv_freq(rope_dim=rope_dim) if rope_dim else None
    q = g[:, :Hq] if Hq else None
    q_out, k_hat, v_hat = fm.fm_kv4_append(
        g[:, Hq:Hq + Hkv], g[:, Hq + Hkv:], kp, vp, dev(table), dev(seq), dev(pos),
        inv_freq=None if freq is None else dev(freq), positions=None if positions is None else dev(positions), q=q,
        q_out=q if q_in_place else None, values=True)
    torch.cuda.synchronize()
    x = qkv.double().numpy()
    at = pos if positions is None else positions
    k = OC.rotate(x[:, Hq:Hq + Hkv], at, freq)
    v = x[:, Hq + Hkv:]
    live = (seq >= 0) & (seq < table.shape[0]) & (pos >= 0) & (pos < table.shape[1] * page)
    want = {"k": start.copy(), "v": start.copy()}
    hat = {}
    with np.errstate(all="ignore"):
        for name, a in (("k", k), ("v", v)):
            codes, scales = OC.quant4(a)
            hat[name] = np.where(live[:, None, None], OC.dequant4(codes, scales), 0.0)
            for t in np.flatnonzero(live):
                p, s = table[seq[t], pos[t] // page], pos[t] % page
                if p < 0 or p >= n_pages:
                    hat[name][t] = 0.0
                    continue
                want[name][p, :, s * 64:(s + 1) * 64] = codes[t]
                want[name][p, :, page * 64 + 4 * s:page * 64 + 4 * s + 4] = scales[t]
    for name, got in (("k", kp), ("v", vp)):  # the new records, and nothing else
        bad = np.argwhere(got.cpu().numpy() != want[name])
        assert bad.size == 0, (name, bad[:5].tolist(), len(bad))
    np.testing.assert_array_equal(k_hat.double().cpu().numpy(), hat["k"])
    np.testing.assert_array_equal(v_hat.double().cpu().numpy(), hat["v"])
    if Hq:
        with np.errstate(all="ignore"):
            ref = OC.rotate(x[:, :Hq], at, freq)
        got = q_out.double().cpu().numpy()
        dead = x[:, :Hq] if q_in_place else np.zeros_like(ref)
        ref = np.where(live[:, None, None], ref, dead)
        tol = half_step(qkv.dtype) * np.abs(ref) * (1 + 2.0 ** -10) + torch.finfo(qkv.dtype).tiny * 2.0 ** -7
        fine = np.isfinite(ref)
        assert (np.isfinite(got) == fine).all()
        assert (np.abs(got - ref)[fine] <= tol[fine]).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,Hq,Hkv,page,rope_dim", [(1, 0, 1, 16, 64), (1, 5, 3, 16, 128), (37, 32, 8, 16, 64),
                                                    (200, 7, 1, 48, 128), (64, 0, 2, 64, 0), (300, 1, 5, 32, 64)])
def test_append_writes_the_exact_records(dtype, T, Hq, Hkv, page, rope_dim):
    rng = np.random.default_rng(T + Hq + page)
    case = append_case(rng, dtype, T, Hq, Hkv, page, rope_dim)
    check_append(*case, Hq, Hkv, page, rope_dim)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_append_far_positions_and_queries_in_place(dtype):
    rng = np.random.default_rng(3)
    qkv, seq, pos, table = append_case(rng, dtype, 50, 4, 2, 16, 64)
    far = rng.integers(0, 1 << 20, 50).astype(np.int64)
    far[:3] = [(1 << 20) - 1, 0, 105615]
    check_append(qkv, seq, pos, table, 4, 2, 16, 64, positions=far, q_in_place=True)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_append_borders_zeros_and_what_is_not_finite(dtype):
    """Values on the borders between codes, all-zero groups, magnitudes at the
    ends of the type, infinities and NaN (their group reads as NaN, its
    neighbours as they are)."""
    rng = np.random.default_rng(4)
    T, Hkv = 24, 2
    x = rng.standard_normal((T, 2 * Hkv, 128))
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 3.0, 4.5])
    x[0] = rng.choice(borders, x[0].shape) * rng.choice([-1, 1], x[0].shape)
    x[1] = 0.0
    x[2] = -0.0
    x[3, :, ::2] = 0.0
    info = torch.finfo(TYPES[dtype])
    x[4] = rng.choice([info.max, -info.max, 1.0], x[4].shape)
    x[5] = rng.choice([info.tiny, -info.tiny, 0.0], x[5].shape)
    x[6, :, 5] = np.nan
    x[7, :, 40] = np.inf
    x[8, :, 127] = -np.inf
    x[9] *= 2.0 ** -12
    x[10] *= 2.0 ** 10
    x[11] = 6.0
    x[12] = 3.0
    qkv = torch.from_numpy(x).to(TYPES[dtype])
    seq = np.zeros(T, np.int32)
    pos = np.arange(T, dtype=np.int64)
    table = np.array([[1, 0]], np.int32)
    check_append(qkv, seq, pos, table, 0, Hkv, 16, 0)
    # rotated: position 0 leaves the numbers, and so their ties, as they are
    check_append(qkv, seq, pos, table, 0, Hkv, 16, 64, positions=np.zeros(T, np.int64))


def test_append_skips_missing_pages_and_positions_past_the_table():
    rng = np.random.default_rng(5)
    qkv = torch.from_numpy(rng.standard_normal((6, 3, 128))).float()
    table = np.array([[0, -1, 9000], [2, 1, 3]], np.int32)
    seq = np.array([0, 0, 0, 1, 1, 1], np.int32)
    pos = np.array([3, 17, 40, 48, -1, 47], np.int64)
    check_append(qkv[:, 1:], seq, pos, np.where(table == 9000, -7, table), 0, 1, 16, 64)
    kp = torch.zeros(4, 1, 16 * 68, device=DEV, dtype=torch.uint8)
    vp = torch.zeros_like(kp)
    g = qkv.to(DEV)
    fm.fm_kv4_append(g[:, 1:2], g[:, 2:], kp, vp, dev(table), dev(seq), dev(np.array([0, 0, 40, 1 << 40, -1, 0])))
    torch.cuda.synchronize()
    assert kp[3].sum() == 0 and kp[1].sum() == 0 and kp[0].sum() > 0 and kp[2].sum() > 0


def test_append_into_a_pool_past_32_bits_and_strided_pools():
    rng = np.random.default_rng(6)
    page, Hkv = 64, 2
    qkv = torch.from_numpy(rng.standard_normal((8, 4, 128))).bfloat16()
    x = qkv.double().numpy()
    codes, scales = OC.quant4(x)
    big = torch.empty(300000, 2, Hkv, page * 68, device=DEV, dtype=torch.uint8)  # 5.2 GB: [page, k or v, head, block]
    kp, vp = big[:, 0], big[:, 1]
    table = np.array([[299999, 7]], np.int32)
    pos = np.arange(60, 68, dtype=np.int64)
    for t in (kp[299999], vp[299999], kp[7], vp[7]):
        t.zero_()
    g = qkv.to(DEV)
    fm.fm_kv4_append(g[:, :2], g[:, 2:], kp, vp, dev(table), dev(np.zeros(8, np.int32)), dev(pos))
    torch.cuda.synchronize()
    for i, pool in enumerate((kp, vp)):
        got = pool[[299999, 7]].cpu().numpy()
        for t in range(8):
            p, s = (0, pos[t]) if pos[t] < 64 else (1, pos[t] - 64)
            np.testing.assert_array_equal(got[p, :, s * 64:s * 64 + 64], codes[t, 2 * i:2 * i + 2])
            np.testing.assert_array_equal(got[p, :, page * 64 + 4 * s:page * 64 + 4 * s + 4], scales[t, 2 * i:2 * i + 2])
    # and the attention that reads them there
    q = torch.from_numpy(rng.standard_normal((1, 1, 4, 128))).bfloat16()
    near = np.concatenate([kp[[299999, 7]].cpu().numpy(), vp[[299999, 7]].cpu().numpy()])
    o = fm.fm_kv4_attention(q.to(DEV), kp, vp, dev(table), dev(np.array([68], np.int32)),
                            kv_start=dev(np.array([60], np.int32)))
    check_attention(o, q, near[:2], near[2:], np.array([[0, 1]], np.int32), [68], page, kv_start=[60])


# --------------------------------------------------------------- the attention


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 100, 257]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 1), (8, 8), (12, 4), (16, 1), (20, 2), (32, 1), (56, 8), (64, 1)])
def test_attention_heads_and_lengths(dtype, Hq, Hkv):
    run_attention(np.random.default_rng(Hq * 10 + Hkv), LENS, Hq, Hkv, dtype=dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("Tq,Hq,Hkv", [(2, 4, 4), (3, 8, 2), (5, 6, 1), (8, 32, 4), (17, 3, 1), (64, 2, 2)])
def test_attention_drafts(dtype, Tq, Hq, Hkv):
    run_attention(np.random.default_rng(Tq), LENS, Hq, Hkv, Tq=Tq, dtype=dtype, page=32)


@pytest.mark.parametrize("page", [16, 48, 64, 1024])
@pytest.mark.parametrize("lens", [[1000, 4096, 1], [5000], [777, 0, 0, 3000]])
def test_attention_longer_rows_and_pages(page, lens):
    rng = np.random.default_rng(page)
    run_attention(rng, lens, 16, 2, page=page, dtype="bf16")
    run_attention(rng, lens, 4, 2, page=page, dtype="fp32", Tq=2)


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
@pytest.mark.parametrize("kw", [
    dict(softcap=20.0), dict(softcap=2.0), dict(window=1), dict(window=5), dict(window=200), dict(kv_start=True),
    dict(slopes=True), dict(softcap=30.0, slopes=True, window=40, kv_start=True), dict(scale=0.0), dict(scale=-0.3),
    dict(scale=1.7, softcap=50.0)], ids=str)
@pytest.mark.parametrize("Tq", [1, 4])
def test_attention_masks_caps_and_biases(dtype, kw, Tq):
    rng = np.random.default_rng(11)
    kw = dict(kw)
    lens = LENS + [900]
    if kw.pop("kv_start", False):
        kw["kv_start"] = [0, 1, 1, 20, 3, -5, 31, 10, 50, 256, 899]
    if kw.pop("slopes", False):
        kw["slopes"] = np.exp2(-np.arange(8.0)).astype(np.float32)
    run_attention(rng, lens, 8, 2, Tq=Tq, dtype=dtype, **kw)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("softcap", [65.0, 300.0, 2.0 ** 17, 2.0 ** 32])
def test_attention_with_a_cap_far_above_the_scores(dtype, softcap):
    """Such a cap costs no accuracy: the tolerance has no term of the cap."""
    rng = np.random.default_rng(12)
    lens, page, kind = [300, 41, 700], 16, TYPES[dtype]
    for spread in (0.3, 3.0):  # scores of a few units, and of hundreds
        kp, vp, table = make_cache(rng, lens, 2, page)
        q = torch.from_numpy(spread * rng.standard_normal((3, 1, 8, 128))).to(kind)
        o = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.asarray(lens, np.int32)), softcap=softcap)
        k, there = OC.read_cache(kp, table, page)
        v, _ = OC.read_cache(vp, table, page)
        ref, _, abs_v, top_v = OC.attention(q.double().numpy(), k, v, there, lens, softcap=softcap)
        _, err_x, _, _ = OC.attention(q.double().numpy(), k, v, there, lens)
        w = (2.0 ** -11 if dtype == "bf16" else 2.0 ** -20) + 2.0 ** -23 * (700 / 16 + 16)
        tol = (2 * 2.0 ** -20 * err_x + w) * abs_v + top_v + half_step(kind) * np.abs(ref) + 1e-37
        assert (np.abs(o.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("max_sel", [1, 7, 64, 300, 1500])
@pytest.mark.parametrize("Hq,Hkv,Tq", [(32, 1, 1), (8, 4, 3)])
def test_attention_over_a_kept_list(dtype, max_sel, Hq, Hkv, Tq):
    """Lists in and out of order, entries twice, outside the row or negative,
    counts of zero and past the list."""
    rng = np.random.default_rng(max_sel)
    lens = [2000, 700, 40, 0, 1999, 5]
    idx = np.stack([rng.integers(-3, max(n, 1) + 20, max_sel) for n in lens]).astype(np.int32)
    idx[0] = np.sort(rng.choice(2000, max_sel, replace=False))
    count = [max_sel, max(1, max_sel // 2), max_sel + 100, max_sel, 0, -4]
    run_attention(rng, lens, Hq, Hkv, Tq=Tq, dtype=dtype, idx=idx, count=count, page=48)
    run_attention(rng, lens, Hq, Hkv, Tq=Tq, dtype=dtype, idx=idx, count=count, window=300,
                  kv_start=[5, 600, 0, 0, 0, 0], softcap=9.0)


def test_attention_missing_pages_are_not_seen():
    rng = np.random.default_rng(13)
    lens = [300, 200, 64]
    kp, vp, table = make_cache(rng, lens, 2, 16)
    table[0, 3] = -1
    table[0, 7] = kp.shape[0]
    table[1, :] = -5
    table[2, 1:] = 1 << 30
    run_attention(rng, lens, 8, 2, cache=(kp, vp, table))
    run_attention(rng, lens, 8, 2, cache=(kp, vp, table), dtype="fp32", Tq=3)
    idx = np.stack([rng.permutation(300)[:100] for _ in lens]).astype(np.int32)
    run_attention(rng, lens, 8, 2, cache=(kp, vp, table), idx=idx, count=[100] * 3)


@pytest.mark.parametrize("listed", [False, True])
def test_attention_is_not_touched_by_what_it_does_not_see(listed):
    """Records past the end, before the start, outside the window and of pages
    that are not listed hold NaN scales: nothing of it reaches the output."""
    rng = np.random.default_rng(14)
    lens, page = [100, 37, 0, 16], 16
    kp, vp, table = make_cache(rng, lens, 2, page, spare=5, cap=160)
    seen = np.zeros((kp.shape[0], page), bool)
    start = [20, 0, 0, 3]
    for b, n in enumerate(lens):
        for j in range(max(start[b], n - 50 + 1 - 1), n):
            seen[table[b, j // page], j % page] = True
    idx = count = None
    if listed:
        idx = np.stack([np.arange(160)] * 4).astype(np.int32)
        count = [160] * 4
    for p in (kp, vp):
        s = p[:, :, page * 64:].reshape(p.shape[0], 2, page, 4)
        s[~np.broadcast_to(seen[:, None], s.shape[:3])] = 255
        p[:, :, page * 64:] = s.reshape(p.shape[0], 2, -1)
    for Tq in (1, 2):
        # a query sees at most 49 positions back of the last one: all of them hold numbers
        run_attention(rng, lens, 4, 2, Tq=Tq, cache=(kp, vp, table), kv_start=start, window=50 - Tq + 1, idx=idx,
                      count=count)


def test_attention_a_seen_nan_makes_its_rows_nan_only():
    rng = np.random.default_rng(15)
    lens, page = [50, 50], 16
    for which in (0, 1):
        kp, vp, table = make_cache(rng, lens, 2, page)
        p = (kp, vp)[which]
        p[table[0, 1], 0, page * 64 + 4 * 3 + 2] = 255  # row 0, position 19, kv head 0, dims 64..95
        q = torch.from_numpy(rng.standard_normal((2, 4, 128))).bfloat16().to(DEV)
        o = fm.fm_kv4_attention(q, dev(kp), dev(vp), dev(table), dev(np.array(lens, np.int32))).float().cpu()
        if which == 0:
            assert torch.isnan(o[0, :2]).all()  # a logit is NaN: so is its softmax
        else:
            assert torch.isnan(o[0, :2, 64:96]).all()
        assert torch.isfinite(o[0, 2:]).all() and torch.isfinite(o[1]).all()


def test_attention_a_nan_reaches_the_queries_that_see_it_only():
    """Drafts, a window and starts: the NaN record lies before, among or after
    what a query sees."""
    rng = np.random.default_rng(16)
    lens, page, Tq = [60, 61], 16, 4
    kp, vp, table = make_cache(rng, lens, 1, page)
    q = torch.from_numpy(rng.standard_normal((2, Tq, 2, 128))).half().to(DEV)
    for at in (30, 57, 59):
        for p in (kp, vp):
            x = p.copy()
            x[table[0, at // 16], 0, page * 64 + 4 * (at % 16)] = 255  # row 0: dims 0..31
            pools = (x, vp) if p is kp else (kp, x)
            for kw in (dict(), dict(window=2), dict(window=28)):
                o = fm.fm_kv4_attention(q, dev(pools[0]), dev(pools[1]), dev(table), dev(np.array(lens, np.int32)),
                                        **kw).float().cpu()
                assert torch.isfinite(o[1]).all()
                for t in range(Tq):
                    pos = 60 - Tq + t
                    sees = at <= pos and pos - at < kw.get("window", 1 << 30)
                    assert bool(torch.isnan(o[0, t, :, :32]).all()) == sees, (at, kw, t)
                    if not sees:
                        assert torch.isfinite(o[0, t]).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lo,hi", [(1, 4), (20, 40), (60, 200), (125, 128), (215, 218)])
def test_attention_scales_far_apart(dtype, lo, hi):
    """Values from 2^-126 to 2^90, alone and mixed in one row (keys kept small
    enough for finite scores)."""
    rng = np.random.default_rng(lo)
    lens, page = [200, 33], 16
    kp, _, table = make_cache(rng, lens, 2, page, lo=max(1, min(lo, 126)), hi=min(hi, 128))
    _, vp, _ = make_cache(rng, lens, 2, page, lo=lo, hi=hi)
    run_attention(rng, lens, 8, 2, cache=(kp, vp, table), dtype=dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_attention_queries_of_any_size(dtype):
    rng = np.random.default_rng(17)
    run_attention(rng, [300, 20], 8, 2, dtype=dtype, q_scale=1e-6)
    run_attention(rng, [300, 20], 8, 2, dtype=dtype, q_scale=200.0)
    kp, vp, table = make_cache(rng, [64], 1, 16)
    q = torch.zeros(1, 4, 128, dtype=TYPES[dtype])
    q[0, 1] = 1.0
    q[0, 2, 5] = 60000.0
    o = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.array([64], np.int32)))
    check_attention(o, q.view(1, 1, 4, 128), kp, vp, table, [64], 16)


def test_attention_strided_queries_and_pools():
    rng = np.random.default_rng(18)
    lens, page = [100, 64, 3], 16
    kp, vp, table = make_cache(rng, lens, 2, page)
    both = dev(np.stack([kp, vp], axis=1))            # [page, k or v, head, block]
    heads = dev(np.stack([kp, vp]).transpose(0, 2, 1, 3))  # [k or v, head, page, block]
    qkv = torch.from_numpy(rng.standard_normal((3 * 2, 12, 128))).half()
    q = qkv.to(DEV).view(3, 2, 12, 128)[:, :, 4:8]
    lens_d = dev(np.array(lens, np.int32))
    wide = dev(np.concatenate([table, table], axis=1))[:, :table.shape[1]]  # rows of a larger table
    a = fm.fm_kv4_attention(q, dev(kp), dev(vp), dev(table), lens_d)
    b = fm.fm_kv4_attention(q, both[:, 0], both[:, 1], wide, lens_d)
    c = fm.fm_kv4_attention(q, heads[0].transpose(0, 1), heads[1].transpose(0, 1), dev(table), lens_d)
    check_attention(a, qkv.view(3, 2, 12, 128)[:, :, 4:8], kp, vp, table, lens, page)
    assert torch.equal(a, b) and torch.equal(a, c)


def test_attention_is_the_same_for_every_bound_and_run():
    """max_len only sizes the launch; the same call gives the same bits."""
    rng = np.random.default_rng(19)
    lens = [3000, 10, 2999]
    kp, vp, table = make_cache(rng, lens, 1, 16, cap=6000)
    q = torch.from_numpy(rng.standard_normal((3, 8, 128))).bfloat16()
    args = (q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.array(lens, np.int32)))
    a = fm.fm_kv4_attention(*args)
    assert torch.equal(a, fm.fm_kv4_attention(*args))
    for bound in (3000, 3001, 4096):
        o = fm.fm_kv4_attention(*args, max_len=bound)
        check_attention(o, q.view(3, 1, 8, 128), kp, vp, table, lens, 16)
    o = fm.fm_kv4_attention(*args, max_len=100)  # longer rows count as the bound
    check_attention(o, q.view(3, 1, 8, 128), kp, vp, table, [100, 10, 100], 16)


@pytest.mark.parametrize("window", [256, 257, 1 << 30, (1 << 31) - 1])
def test_attention_windows_at_and_past_the_row(window):
    rng = np.random.default_rng(22)
    run_attention(rng, [257, 3, 0, 256], 4, 2, Tq=2, window=window)
    run_attention(rng, [257, 3, 0, 256], 4, 2, Tq=2, window=window, kv_start=[(1 << 31) - 1, 0, 7, 100])


@pytest.mark.parametrize("B", [33, 200])
def test_attention_many_rows_share_their_ctas(B):
    """More rows than lanes find their places by the block's scan; short and long
    rows share CTAs, and rows of nothing still get their zeros."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 700, B)
    lens[::7] = 0
    lens[5] = 1500
    run_attention(rng, [int(n) for n in lens], 2, 2, dtype="fp32")
    run_attention(rng, [int(n) for n in lens], 12, 1, dtype="bf16", Tq=2, page=64)
    run_attention(rng, [int(min(n, 400)) for n in lens], 2, 1)  # short enough for a CTA a unit


def test_attention_one_long_row_over_all_ctas():
    """One kv head: every CTA has a part of the only unit, or of the two units of
    a second tile of query rows."""
    rng = np.random.default_rng(23)
    for Hq in (4, 20):
        run_attention(rng, [60000], Hq, 1, page=128)
        run_attention(rng, [40001], Hq, 1, page=48, dtype="fp32")


def test_attention_workspace_is_enough_and_not_overrun():
    rng = np.random.default_rng(20)
    lens = [2500, 1300]
    kp, vp, table = make_cache(rng, lens, 2, 16)
    q = torch.from_numpy(rng.standard_normal((2, 2, 20, 128))).bfloat16()
    c = fm._kv4_cache(dev(kp), dev(vp), dev(table))
    d = fm.fm_kv4_attn_desc(1, 2, 20, 16, 2560, 16, 16, None, table.shape[1] * 16, None, None, 0, 0.1, 0.0, None, 0)
    import ctypes
    need = fm.lib().fm_kv4_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(d))
    ws = torch.full((need + 512,), 0xA5, device=DEV, dtype=torch.uint8)  # 0xA5 bytes are large negative floats
    out = torch.full((2, 2, 20, 128), 7.0, device=DEV, dtype=torch.bfloat16)
    o = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.array(lens, np.int32)), out=out,
                            workspace=ws[:need])
    assert o.data_ptr() == out.data_ptr() and bool((ws[need:] == 0xA5).all())
    check_attention(o, q, kp, vp, table, lens, 16)


def test_attention_graphs_streams_and_calls_at_once():
    """Two captured graphs and eager calls on two streams, replayed and run in
    turn and at once: each has its own workspace, and replays read the buffers'
    newest contents."""
    rng = np.random.default_rng(21)
    sets, graphs = [], []
    for i, lens in enumerate(([2000, 100], [64, 1500])):
        kp, vp, table = make_cache(rng, lens, 2, 16)
        q = torch.from_numpy(rng.standard_normal((2, 1, 8, 128))).bfloat16()
        sets.append((q, kp, vp, table, lens, [q.to(DEV), dev(kp), dev(vp), dev(table), dev(np.array(lens, np.int32))]))
    fm.fm_kv4_attention(*sets[0][5])
    torch.cuda.synchronize()
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = fm.fm_kv4_attention(*s[5])
        graphs.append((g, o))
    for g, _ in graphs:
        g.replay()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for rep in range(3):
        for s, st, (g, _) in zip(sets, streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
            outs.append((s, fm.fm_kv4_attention(*s[5], stream=streams[1 - streams.index(st)])))
    torch.cuda.synchronize()
    for s, (g, o) in zip(sets, graphs):
        check_attention(o, s[0], s[1], s[2], s[3], s[4], 16)
        for t, e in outs:
            if t is s:
                assert torch.equal(e, o)
    # new queries in the captured buffer
    q2 = torch.from_numpy(rng.standard_normal((2, 1, 8, 128))).bfloat16()
    sets[0][5][0].copy_(q2)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    check_attention(graphs[0][1], q2, sets[0][1], sets[0][2], sets[0][3], sets[0][4], 16)


def test_empty_calls():
    pages = torch.zeros(2, 1, 16 * 68, device=DEV, dtype=torch.uint8)
    table = torch.zeros(1, 1, device=DEV, dtype=torch.int32)
    z = torch.zeros(0, 1, 128, device=DEV)
    q_out, k_hat, v_hat = fm.fm_kv4_append(z, z, pages, pages.clone(), table, torch.zeros(0, device=DEV).int(),
                                           torch.zeros(0, device=DEV).long(), values=True)
    assert k_hat.shape == (0, 1, 128)
    o = fm.fm_kv4_attention(torch.zeros(0, 1, 128, device=DEV), pages, pages, table[:0], torch.zeros(0, device=DEV).int())
    assert o.shape == (0, 1, 128)
    s, c, k = fm.fm_add_rmsnorm_fp8(torch.zeros(0, 256, device=DEV))
    assert c.shape == (0, 256) and k.shape == (0, 2)
    with pytest.raises(ValueError):
        fm.fm_kv4_attention(torch.zeros(1, 1, 128, device=DEV), pages, pages, table, torch.zeros(1).int())


# -------------------------------------------------------------- indexer keys


def records(comp_k):
    """[..., 132] bytes -> (values of the codes, scales) in fp64."""
    r = comp_k.cpu().numpy()
    return O.e4m3_decode(r[..., :128]).astype(np.float64), np.ascontiguousarray(r[..., 128:]).view(np.float32)[..., 0].astype(np.float64)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,L,rope_dim,hadamard", [(1, 1, 64, True), (5, 3, 64, True), (33, 2, 0, True),
                                                   (100, 4, 128, False), (257, 3, 0, False)])
def test_index_records_match_the_oracle(dtype, T, L, rope_dim, hadamard):
    """A code is off by half a step of e4m3 (2^-4 of the value, 2^-10 of the
    scale among the subnormals), the transform's fp32 sums by 2^-20 of the
    scale's range."""
    rng = np.random.default_rng(T + L)
    B, N = 3, 256
    k = torch.from_numpy(rng.standard_normal((T, L, 128)) * np.exp2(rng.integers(-9, 9, (T, L, 1)))).to(TYPES[dtype])
    slots = rng.permutation(B * N)[:T]
    row, chunk = (slots // N).astype(np.int32), (slots % N).astype(np.int32)
    pad = rng.random(T) < 0.1
    pad[0] = False
    row[pad & (np.arange(T) % 2 == 0)] = -1
    chunk[pad & (np.arange(T) % 2 == 1)] = N
    positions = rng.integers(0, 1 << 20, T).astype(np.int64)
    freq = O.yarn_inv_freq(rope_dim=rope_dim) if rope_dim else None
    comp_k = [torch.full((B, N, 132), 0x11, device=DEV, dtype=torch.uint8) for _ in range(L)]
    fm.fm_index_append(k.to(DEV), comp_k, dev(row), dev(chunk), inv_freq=None if freq is None else dev(freq),
                       positions=dev(positions) if rope_dim else None, hadamard=hadamard)
    torch.cuda.synchronize()
    x = OC.index_vector(k.double().numpy(), positions, freq, hadamard)
    for l in range(L):
        codes, scale = records(comp_k[l])
        touched = np.zeros((B, N), bool)
        for t in np.flatnonzero(~pad):
            b, n = row[t], chunk[t]
            touched[b, n] = True
            want = np.abs(x[t, l]).max() / 448
            assert abs(scale[b, n] - want) <= 2.0 ** -20 * want
            got = codes[b, n] * scale[b, n]
            tol = np.maximum(2.0 ** -4 * np.abs(x[t, l]), 2.0 ** -10 * want) + 2.0 ** -20 * 448 * want
            assert (np.abs(got - x[t, l]) <= tol).all()
        rest = comp_k[l].cpu().numpy()[~touched]
        assert (rest == 0x11).all()  # every other record as it was


def test_index_records_of_zeros_tiny_and_not_finite_keys():
    k = torch.zeros(6, 1, 128)
    k[1] = 1e-42
    k[2, 0, 3] = float("nan")
    k[3, 0, 7] = float("inf")
    k[4] = 3e38
    k[5, 0, 0] = -1.0
    comp_k = [torch.zeros(1, 8, 132, device=DEV, dtype=torch.uint8)]
    fm.fm_index_append(k.to(DEV), comp_k, dev(np.zeros(6, np.int32)), dev(np.arange(6, dtype=np.int32)), hadamard=False)
    codes, scale = records(comp_k[0])
    v = codes[0] * scale[0][:, None]
    assert (v[0] == 0).all() and scale[0, 0] == 0
    assert (v[1] == 0).all() and scale[0, 1] == 0
    assert np.isnan(v[2]).all() and np.isnan(v[3]).all()
    np.testing.assert_allclose(v[4], 3e38, rtol=2.0 ** -4)
    assert v[5, 0] == pytest.approx(-1.0, rel=2.0 ** -22) and (v[5, 1:] == 0).all()


# -------------------------------------------------------------------- the norm


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,H", [(1, 128), (3, 256), (7, 4096), (5, 7168), (2, 8320), (2, 16384), (1, 32768), (300, 512), (40, 1152)])
@pytest.mark.parametrize("per_row", [False, True])
def test_norm_matches_the_oracle(dtype, T, H, per_row):
    """fp32 sums: the mean's and the scale's error is 2^-20 (H terms, each
    rounded, summed in a tree); codes half a step of e4m3 beside it."""
    rng = np.random.default_rng(T * H)
    kind = TYPES[dtype]
    x = torch.from_numpy(rng.standard_normal((T, H)) * np.exp2(rng.integers(-6, 7, (T, 1)))).to(kind)
    r = torch.from_numpy(rng.standard_normal((T, H))).to(kind)
    gain = torch.from_numpy(1 + 0.1 * rng.standard_normal(H)).to(kind)
    for res, g in ((r, gain), (None, gain), (r, None)):
        s, codes, scales = fm.fm_add_rmsnorm_fp8(x.to(DEV), None if res is None else res.to(DEV),
                                                 None if g is None else g.to(DEV), group=H if per_row else 128)
        torch.cuda.synchronize()
        z, y = OC.add_rmsnorm(x.double().numpy(), None if res is None else res.double().numpy(),
                              None if g is None else g.double().numpy())
        tol = half_step(kind) * np.abs(z) * (1 + 2.0 ** -10) + 2.0 ** -24 * np.abs(z) + torch.finfo(kind).tiny * 2.0 ** -9
        assert (np.abs(s.double().cpu().numpy() - z) <= tol).all()
        group = H if per_row else 128
        want = np.abs(y.reshape(T, -1, group)).max(-1) / 448
        sc = scales.double().cpu().numpy()
        assert (np.abs(sc - want) <= 2.0 ** -18 * want).all()
        got = codes.float().double().cpu().numpy() * np.repeat(sc, group, axis=1)
        wide = np.repeat(want, group, axis=1)
        assert (np.abs(got - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * wide) + 2.0 ** -18 * np.abs(y)
                + 2.0 ** -22 * 448 * wide).all()


def test_norm_in_place_strided_and_odd_rows():
    rng = np.random.default_rng(31)
    big = torch.from_numpy(rng.standard_normal((6, 3, 512))).float().to(DEV)
    x, r = big[:, 0], big[:, 2]
    want = fm.fm_add_rmsnorm_fp8(x.contiguous(), r.contiguous())
    got = fm.fm_add_rmsnorm_fp8(x, r)
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for which in (0, 1):
        a, b = x.clone(), r.clone()
        s, c, k = fm.fm_add_rmsnorm_fp8(a, b, sum_out=(a, b)[which])
        assert s.data_ptr() == (a, b)[which].data_ptr()
        assert torch.equal(s, want[0]) and torch.equal(c.view(torch.uint8), want[1].view(torch.uint8))
    # zeros, a NaN, an infinity, and the largest values
    z = torch.zeros(5, 256, device=DEV)
    z[1, 200] = float("nan")
    z[2, 5] = float("inf")
    z[3] = 1e18
    z[4, 130] = 2.0
    s, c, k = fm.fm_add_rmsnorm_fp8(z)
    k = k.cpu()
    assert (k[0] == 0).all() and (c[0].float() == 0).all()
    assert torch.isnan(k[1]).all() and torch.isnan(k[2]).all()
    v = c.float().cpu() * k.repeat_interleave(128, dim=1)
    torch.testing.assert_close(v[3], torch.ones(256), rtol=2.0 ** -20, atol=0)
    assert k[4, 0] == 0 and v[4, 130] == pytest.approx(2.0 / math.sqrt(4.0 / 256 + 1e-6), rel=2.0 ** -18)


@pytest.mark.parametrize("group", [128, 256])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_norm_without_eps_of_zeros_is_zeros(dtype, group):
    z = torch.zeros(2, 256, device=DEV, dtype=TYPES[dtype])
    z[1, 7] = 4.0
    s, c, k = fm.fm_add_rmsnorm_fp8(z, eps=0.0, group=group)
    assert torch.equal(s, z) and (c[0].float() == 0).all() and (k[0] == 0).all()
    assert float(c[1, 7]) * float(k[1, 0]) == pytest.approx(16.0, rel=2.0 ** -18) and (k[1, 1:] == 0).all()


# -------------------------------------------------------------- a run of them


def test_a_decode_step_from_the_hidden_state_to_the_output():
    """The operators as a serving loop uses them: the residual norm, a prompt's
    and then a step's keys, values and indexer keys appended, the retriever's
    scores and top-K over the records that were appended, and the attention
    over the kept positions only."""
    rng = np.random.default_rng(41)
    B, N, page, Hq, Hkv, keep = 3, 320, 16, 16, 2, 64
    n0 = [300, 150, 40]
    weights = H.G.make_weights(411, 3)
    r = fm.Retriever(weights, device=0, max_batch=8)
    try:
        per = N // page
        table = torch.from_numpy(rng.permutation(B * per).reshape(B, per).astype(np.int32)).to(DEV)
        kp = torch.zeros(B * per, Hkv, page * 68, device=DEV, dtype=torch.uint8)
        vp = torch.zeros_like(kp)
        comp_k = [torch.zeros(B, N, 132, device=DEV, dtype=torch.uint8) for _ in range(3)]
        freq = fm.fm_rope_frequencies(DEV)
        lens = np.array(n0)
        store_k, store_i = [[] for _ in range(B)], [[] for _ in range(B)]
        store_v = [[] for _ in range(B)]

        def append(seq, pos):
            T = len(seq)
            qkv = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hkv, 128))).bfloat16()
            ik = torch.from_numpy(rng.standard_normal((T, 3, 128))).bfloat16()
            g = qkv.to(DEV)
            seq_d, pos_d = dev(np.asarray(seq, np.int32)), dev(np.asarray(pos, np.int64))
            q, kh, vh = fm.fm_kv4_append(g[:, Hq:Hq + Hkv], g[:, Hq + Hkv:], kp, vp, table, seq_d, pos_d,
                                         inv_freq=freq, q=g[:, :Hq], values=True)
            fm.fm_index_append(ik.to(DEV), comp_k, seq_d, pos_d.int(), inv_freq=freq, positions=4 * pos_d)
            kh, vh = kh.double().cpu().numpy(), vh.double().cpu().numpy()
            for t, b in enumerate(seq):
                store_k[b].append(kh[t])
                store_v[b].append(vh[t])
            return q

        append([b for b in range(B) for _ in range(n0[b])], [j for b in range(B) for j in range(n0[b])])
        hidden = torch.from_numpy(rng.standard_normal((B, 4096))).float().to(DEV)
        for step in range(3):
            hidden, codes, scales = fm.fm_add_rmsnorm_fp8(hidden, 0.1 * hidden)
            x = codes.float() * scales.repeat_interleave(128, dim=1)  # what the projections would read
            q = append(list(range(B)), lens.tolist())
            lens = lens + 1
            nv = dev(lens.astype(np.int32))
            ens, mask, _ = r.retrieve(x.contiguous(), comp_k, dev(4 * lens.astype(np.int64)), nv, "max", keep)
            r.fm_sync_status()
            H.check_topk_against_rule(mask.cpu().numpy(), ens.cpu().numpy(), lens, keep)
            idx, count = fm.fm_compact_mask(mask, keep)
            o = fm.fm_kv4_attention(q, kp, vp, table, nv, idx=idx, count=count, softcap=40.0)
            k = np.zeros((B, Hkv, N, 128))
            v = np.zeros((B, Hkv, N, 128))
            for b in range(B):
                k[b, :, :lens[b]] = np.stack(store_k[b], 1)
                v[b, :, :lens[b]] = np.stack(store_v[b], 1)
            ref, err_x, abs_v, top_v = OC.attention(q.double().cpu().numpy()[:, None], k, v, np.ones((B, N), bool), lens,
                                             softcap=40.0, idx=idx.cpu().numpy(), count=count.cpu().numpy())
            tol = (2 * 2.0 ** -20 * err_x + 2.0 ** -11 + 2.0 ** -18) * abs_v + top_v + 2.0 ** -8 * np.abs(ref)
            assert (np.abs(o.double().cpu().numpy()[:, None] - ref) <= tol).all()
    finally:
        r.close()


# ------------------------------------------------------------------ in place


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,H", [(9, 128), (5, 512), (300, 1024), (33, 2048), (17, 4096), (5, 8192), (3, 16384), (2, 32768)])
def test_norm_into_its_operands_is_the_norm(dtype, T, H):
    """Every width of row, the sum written over x or over the residual."""
    rng = np.random.default_rng(H)
    x, r = (torch.from_numpy(rng.standard_normal((T, H))).to(TYPES[dtype]).to(DEV) for _ in range(2))
    g = torch.from_numpy(1 + 0.1 * rng.standard_normal(H)).to(TYPES[dtype]).to(DEV)
    for group in (128, H):
        want = fm.fm_add_rmsnorm_fp8(x, r, g, group=group)
        for which in (0, 1):
            ops = [x.clone(), r.clone()]
            got = fm.fm_add_rmsnorm_fp8(*ops, g, group=group, sum_out=ops[which])
            assert got[0].data_ptr() == ops[which].data_ptr()
            for a, b in zip(want, got):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,Hq,Hkv,rope_dim", [(1, 3, 1, 64), (64, 64, 8, 64), (40, 5, 2, 128), (3000, 32, 8, 128)])
def test_queries_rotated_in_place_are_the_rotated_queries(dtype, T, Hq, Hkv, rope_dim):
    rng = np.random.default_rng(T)
    qkv = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hkv, 128))).to(TYPES[dtype]).to(DEV)
    pages = torch.zeros(T // 16 + 1, Hkv, 16 * 68, device=DEV, dtype=torch.uint8)
    table = torch.arange(T // 16 + 1, device=DEV, dtype=torch.int32).view(1, -1)
    seq, pos = torch.zeros(T, device=DEV, dtype=torch.int32), torch.arange(T, device=DEV)
    freq = dev(O.yarn_inv_freq(rope_dim=rope_dim))
    outs = []
    for in_place in (False, True):
        g, kp, vp = qkv.clone(), pages.clone(), pages.clone()
        q = g[:, :Hq]
        o, _, _ = fm.fm_kv4_append(g[:, Hq:Hq + Hkv], g[:, Hq + Hkv:], kp, vp, table, seq, pos, inv_freq=freq, q=q,
                                   q_out=q if in_place else None)
        outs.append((o.clone(), kp, vp))
        assert torch.equal(g[:, Hq:], qkv[:, Hq:])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,Hq,Hkv,Tq", [([300, 20, 0], 8, 2, 1), ([5000, 4000, 17], 8, 2, 1), ([5000, 4000, 17], 24, 2, 3)])
def test_attention_into_its_queries_is_the_attention(dtype, lens, Hq, Hkv, Tq):
    rng = np.random.default_rng(51)
    kp, vp, table = (dev(x) for x in make_cache(rng, lens, Hkv, 16))
    q = torch.from_numpy(rng.standard_normal((len(lens), Tq, Hq, 128))).to(TYPES[dtype]).to(DEV)
    n = dev(np.asarray(lens, np.int32))
    want = fm.fm_kv4_attention(q, kp, vp, table, n)
    got = q.clone()
    fm.fm_kv4_attention(got, kp, vp, table, n, out=got)
    assert torch.equal(want, got)


# ------------------------------------------------ where fp32's range ends


def test_keys_at_the_end_of_fp32():
    """Indexer keys up to 2^120 have their records, whatever the transform adds up; a transform past fp32's range
    gives a NaN scale.  A rotated key past it makes its group NaN, an unrotated one is held to 6 * 2^125."""
    k = torch.zeros(3, 1, 128)
    k[0] = 2.0 ** 120
    k[1] = 2.0 ** 120 * torch.from_numpy(np.random.default_rng(61).choice([-1.0, 1.0], 128)).float()
    k[2] = 2.0 ** 122
    comp_k = [torch.zeros(1, 8, 132, device=DEV, dtype=torch.uint8)]
    fm.fm_index_append(k.to(DEV), comp_k, dev(np.zeros(3, np.int32)), dev(np.arange(3, dtype=np.int32)))
    codes, scale = records(comp_k[0])
    for t in range(2):
        x = OC.index_vector(k[t:t + 1].double().numpy())[0, 0]
        want = np.abs(x).max() / 448
        assert abs(scale[0, t] - want) <= 2.0 ** -20 * want
        tol = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * want) + 2.0 ** -20 * 448 * want
        assert (np.abs(codes[0, t] * scale[0, t] - x) <= tol).all()
    assert np.isnan(scale[0, 2])
    x = torch.zeros(2, 2, 128)
    x[:, :, 64:] = 3e38
    x[:, :, 96:] *= -1
    x[1] *= 2.0 ** -1
    kp, vp = (torch.zeros(1, 1, 16 * 68, device=DEV, dtype=torch.uint8) for _ in range(2))
    g = x.to(DEV)
    # every pair turned by an eighth: a c - b s = 3e38 * 2^(1/2), b c + a s = 0
    _, kh, vh = fm.fm_kv4_append(g[:, :1], g[:, 1:], kp, vp, dev(np.zeros((1, 1), np.int32)), dev(np.zeros(2, np.int32)),
                                 dev(np.arange(2)), inv_freq=dev(np.full(32, math.pi / 4)), positions=dev(np.ones(2, np.int64)),
                                 values=True)
    kh, vh = kh.double().cpu().numpy(), vh.double().cpu().numpy()
    assert np.isnan(kh[0, 0, 64:96]).all() and (np.abs(kh[0, 0, :64]) == 0).all()
    assert (kh[1, 0, 64:96] == 4 * 2.0 ** 125).all()  # 2.1e38 = 4.99 * 2^125
    assert (vh[0, 0, 64:96] == 6 * 2.0 ** 125).all() and (vh[0, 0, 96:] == -6 * 2.0 ** 125).all()


# ------------------------------------------------------- chunks of tokens


@pytest.mark.parametrize("s", [1, 4])
def test_kept_chunks_as_the_positions_that_they_cover(s):
    """A mask over chunks of s tokens, compacted, spread to cache positions and attended to; the last chunk is cut by
    the row's length, and the newest token, in no chunk yet, is listed by the caller."""
    rng = np.random.default_rng(71)
    N, keep_n = 60, 24
    n_chunks = np.array([50, 13, 0])
    lens = [50 * s + 1, 13 * s - s // 2, 1]
    kp, vp, table = make_cache(rng, lens, 2, 16, cap=N * s + 1)
    keep = np.zeros((3, N), np.uint8)
    for b, n in enumerate(n_chunks):
        keep[b, rng.permutation(n)[:min(keep_n, n)]] = 1
    idx, count = fm.fm_compact_mask(dev(keep), keep_n)
    at = (idx[:, :, None] * s + torch.arange(s, device=DEV, dtype=torch.int32)).flatten(1)
    n = dev(np.asarray(lens, np.int32))
    new = torch.where(torch.tensor([True, False, True], device=DEV), n - 1, -1)
    at = torch.cat([new.view(3, 1), at], dim=1).contiguous()
    q = torch.from_numpy(rng.standard_normal((3, 1, 8, 128))).bfloat16()
    o = fm.fm_kv4_attention(q.to(DEV), dev(kp), dev(vp), dev(table), n, idx=at, count=count * s + 1)
    want = np.full((3, N * s + 1), -1)
    total = np.zeros(3, int)
    for b in range(3):
        seen = [c * s + i for c in np.flatnonzero(keep[b]) for i in range(s)] + ([lens[b] - 1] if b != 1 else [])
        want[b, :len(seen)], total[b] = seen, len(seen)
    check_attention(o, q, kp, vp, table, lens, 16, idx=want, count=total)


# ------------------------------------------------ captured, and on another stream


def test_a_whole_step_captured_and_on_another_stream():
    """Norm, appends and attention as one graph, replayed with new inputs and positions, and the same calls on a
    stream of the caller's: all give the bits of the eager step."""
    rng = np.random.default_rng(81)
    B, N, Hq, Hkv, page = 3, 64, 16, 2, 16
    freq = fm.fm_rope_frequencies(DEV)
    table = torch.from_numpy(rng.permutation(B * N // page).reshape(B, -1).astype(np.int32)).to(DEV)
    seq = torch.arange(B, device=DEV, dtype=torch.int32)

    def fresh():
        return [torch.zeros(B * N // page, Hkv, page * 68, device=DEV, dtype=torch.uint8) for _ in range(2)] + [
            torch.zeros(B, N, 132, device=DEV, dtype=torch.uint8) for _ in range(3)]

    x, r = torch.zeros(B, 1024, device=DEV), torch.zeros(B, 1024, device=DEV)
    qkv = torch.zeros(B, Hq + 2 * Hkv, 128, device=DEV, dtype=torch.bfloat16)
    ik = torch.zeros(B, 3, 128, device=DEV, dtype=torch.bfloat16)
    pos = torch.zeros(B, device=DEV, dtype=torch.int64)

    def step(state, stream=None):
        kp, vp, *comp = state
        z, codes, scales = fm.fm_add_rmsnorm_fp8(x, r, stream=stream)
        q, kh, vh = fm.fm_kv4_append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], kp, vp, table, seq, pos, inv_freq=freq,
                                     q=qkv[:, :Hq], values=True, stream=stream)
        if stream is None:
            chunk, n = pos.int(), (pos + 1).int()
        else:
            with torch.cuda.stream(stream):
                chunk, n = pos.int(), (pos + 1).int()
        fm.fm_index_append(ik, comp, seq, chunk, inv_freq=freq, positions=pos, stream=stream)
        return z, codes, scales, q, kh, vh, fm.fm_kv4_attention(q, kp, vp, table, n, stream=stream)

    eager, graphed, aside = fresh(), fresh(), fresh()
    step(fresh())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(graphed)
    for t in graphed:
        t.zero_()
    side = torch.cuda.Stream()
    for i in range(6):
        for t, shape in ((x, x.shape), (r, r.shape), (qkv, qkv.shape), (ik, ik.shape)):
            t.copy_(torch.from_numpy(rng.standard_normal(shape)))
        pos.fill_(5 * i)
        want = step(eager)
        g.replay()
        side.wait_stream(torch.cuda.current_stream())
        got = step(aside, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for a, b, c in zip(want, out, got):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
            assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))
        for a, b, c in zip(eager, graphed, aside):
            assert torch.equal(a, b) and torch.equal(a, c)
