"""The operators around the 4-bit paged cache without a GPU: what the C calls
and the binding refuse before anything is launched, the workspace's size, and
pins of the oracle that the GPU tests use."""
import ctypes
import os

import numpy as np
import pytest
import torch

import oracle.cache as OC
import oracle.retriever as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if not os.path.exists(os.path.join(ROOT, "learned_kv_chunk_b200", "lib", "libfm.so")):
    pytest.skip("libfm.so is not built (python -m learned_kv_chunk_b200.build)", allow_module_level=True)

from learned_kv_chunk_b200 import fm  # noqa: E402

INVALID, ALIGN, UNSUP = 1, 2, 3
FAKE = 0x10000  # never dereferenced: every call below fails its checks first


def cache(**kw):
    d = dict(k_pages=FAKE, v_pages=FAKE, page_stride_bytes=8 * 16 * 68, head_stride_bytes=16 * 68, n_pages=10,
             page_size=16, n_kv_heads=8, B=2, max_pages=4, page_table_stride=4, page_table=FAKE)
    d.update(kw)
    return fm.fm_kv4_cache(**d)


def append_desc(**kw):
    d = dict(dtype=1, T=3, n_q_heads=0, k=FAKE, v=FAKE, q=None, k_stride=1024, v_stride=1024, q_stride=0,
             q_out_stride=0, seq=FAKE, pos=FAKE, positions=None, inv_freq=FAKE, rope_dim=64, q_out=None, k_hat=None,
             v_hat=None)
    d.update(kw)
    return fm.fm_kv4_append_desc(**d)


def attn_desc(**kw):
    d = dict(dtype=1, Tq=1, n_q_heads=32, q=FAKE, q_stride=4096, out=FAKE, kv_len=FAKE, kv_start=None, max_len=64,
             idx=None, count=None, max_sel=0, scale=0.1, softcap=0.0, slopes=None, window=0)
    d.update(kw)
    return fm.fm_kv4_attn_desc(**d)


BAD_CACHES = [
    (dict(k_pages=None), INVALID), (dict(v_pages=None), INVALID), (dict(page_table=None), INVALID),
    (dict(n_pages=0), INVALID), (dict(n_kv_heads=0), INVALID), (dict(n_kv_heads=2000), INVALID), (dict(B=0), INVALID),
    (dict(B=70000), INVALID), (dict(max_pages=0), INVALID), (dict(max_pages=1 << 28), INVALID),
    (dict(page_size=0), UNSUP), (dict(page_size=24), UNSUP), (dict(page_size=2048), UNSUP),
    (dict(page_table_stride=3), INVALID), (dict(k_pages=FAKE + 8), ALIGN), (dict(v_pages=FAKE + 4), ALIGN),
    (dict(page_stride_bytes=8 * 16 * 68 + 8), ALIGN), (dict(head_stride_bytes=16 * 68 + 4), ALIGN),
    (dict(page_table=FAKE + 2), ALIGN),
    (dict(page_stride_bytes=16 * 68), INVALID),  # the heads' blocks would overlap the next page
    (dict(head_stride_bytes=16 * 64), INVALID),  # a block does not fit
    (dict(page_stride_bytes=1 << 60), INVALID),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES, ids=[str(k) for k, _ in BAD_CACHES])
def test_bad_caches_are_refused(kw, status):
    c = cache(**kw)
    a, t = append_desc(), attn_desc()
    assert fm.lib().fm_kv4_append(ctypes.byref(c), ctypes.byref(a), None) == status
    assert fm.lib().fm_kv4_attention(ctypes.byref(c), ctypes.byref(t), FAKE, 1 << 30, None) == status
    assert fm.lib().fm_kv4_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(t)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(seq=None), INVALID), (dict(pos=None), INVALID),
    (dict(T=0), INVALID), (dict(T=(1 << 30) + 1), INVALID), (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(k_stride=1016), INVALID),
    (dict(v_stride=0), INVALID), (dict(rope_dim=32), UNSUP), (dict(inv_freq=None), INVALID),
    (dict(q=FAKE, n_q_heads=32, q_stride=4096, q_out_stride=4096), INVALID),  # no q_out
    (dict(q=FAKE, q_out=FAKE + 4096, n_q_heads=0, q_stride=4096, q_out_stride=4096), INVALID),
    (dict(q=FAKE, q_out=FAKE + 4096, n_q_heads=32, q_stride=4000, q_out_stride=4096), INVALID),
    (dict(q=FAKE, q_out=FAKE, n_q_heads=32, q_stride=4096, q_out_stride=8192), INVALID),  # in place, other strides
    (dict(k=FAKE + 2), ALIGN), (dict(k_stride=1025), ALIGN), (dict(seq=FAKE + 2), ALIGN), (dict(pos=FAKE + 4), ALIGN),
    (dict(positions=FAKE + 4), ALIGN), (dict(inv_freq=FAKE + 4), ALIGN), (dict(k_hat=FAKE + 8), ALIGN),
    (dict(v_hat=FAKE + 8), ALIGN),
])
def test_bad_appends_are_refused(kw, status):
    c, d = cache(), append_desc(**kw)
    assert fm.lib().fm_kv4_append(ctypes.byref(c), ctypes.byref(d), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(kv_len=None), INVALID), (dict(dtype=7), INVALID),
    (dict(Tq=0), INVALID), (dict(Tq=65), UNSUP), (dict(n_q_heads=0), INVALID), (dict(n_q_heads=12), INVALID),
    (dict(n_q_heads=2048), INVALID), (dict(q_stride=4000), INVALID), (dict(max_len=0), INVALID),
    (dict(max_len=65), INVALID), (dict(idx=FAKE, max_sel=8), INVALID), (dict(idx=FAKE, count=FAKE, max_sel=0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(softcap=-1.0), INVALID),
    (dict(softcap=float("nan")), INVALID), (dict(window=-1), INVALID), (dict(q=FAKE + 8), ALIGN),
    (dict(out=FAKE + 8), ALIGN), (dict(q_stride=4097), ALIGN), (dict(kv_len=FAKE + 1), ALIGN),
    (dict(kv_start=FAKE + 1), ALIGN), (dict(slopes=FAKE + 2), ALIGN),
    (dict(idx=FAKE + 2, count=FAKE, max_sel=4), ALIGN),
])
def test_bad_attention_calls_are_refused(kw, status):
    c, d = cache(), attn_desc(**kw)
    assert fm.lib().fm_kv4_attention(ctypes.byref(c), ctypes.byref(d), FAKE, 1 << 40, None) == status


@pytest.mark.parametrize("kw,ok", [
    (dict(scale=2.0 ** 32), True), (dict(scale=-2.0 ** 32), True), (dict(scale=2.0 ** 33), False),
    (dict(scale=-2.0 ** 33), False), (dict(softcap=2.0 ** 32), True), (dict(softcap=2.0 ** -32), True),
    (dict(softcap=2.0 ** 33), False), (dict(softcap=2.0 ** -33), False), (dict(softcap=float("inf")), False)])
def test_attention_scales_and_caps_out_of_range_are_refused(kw, ok):
    c, d = cache(), attn_desc(**kw)
    assert (fm.lib().fm_kv4_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(d)) > 0) == ok
    if not ok:
        assert fm.lib().fm_kv4_attention(ctypes.byref(c), ctypes.byref(d), FAKE, 1 << 40, None) == INVALID


def test_attention_workspace_rules():
    c, d = cache(), attn_desc()
    need = fm.lib().fm_kv4_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(d))
    assert need > 0
    f = fm.lib().fm_kv4_attention
    assert f(ctypes.byref(c), ctypes.byref(d), None, need, None) == INVALID
    assert f(ctypes.byref(c), ctypes.byref(d), FAKE, need - 1, None) == INVALID
    assert f(ctypes.byref(c), ctypes.byref(d), FAKE + 8, need, None) == ALIGN
    # the size is bounded by a constant times the work: one long row, and many
    for B, pages in ((1, 1 << 16), (64, 1 << 12), (65535, 4)):
        c = cache(B=B, max_pages=pages, page_table_stride=pages)
        d = attn_desc(max_len=pages * 16)
        n = fm.lib().fm_kv4_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(d))
        assert 0 < n <= 32 * 130 * 4 * max(4096, 8 * B) + 256, (B, pages, n)


def test_bad_index_appends_are_refused():
    f = fm.lib().fm_index_append
    arr = (ctypes.c_void_p * 3)(FAKE, FAKE, FAKE)

    def call(k=FAKE, dtype=0, stride=384, T=5, L=3, row=FAKE, chunk=FAKE, positions=FAKE, freq=FAKE, rd=64, had=1,
             keys=arr, row_stride=132 * 8, B=2, N=8):
        return f(k, dtype, stride, T, L, row, chunk, positions, freq, rd, had, keys, row_stride, B, N, None)

    for kw, status in [(dict(k=None), INVALID), (dict(row=None), INVALID), (dict(chunk=None), INVALID),
                       (dict(keys=None), INVALID), (dict(T=0), INVALID), (dict(T=2147483647), INVALID), (dict(L=0), INVALID), (dict(L=5), INVALID),
                       (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(dtype=9), INVALID), (dict(rd=48), UNSUP),
                       (dict(positions=None), INVALID), (dict(freq=None), INVALID), (dict(stride=380), INVALID),
                       (dict(row_stride=132 * 7), INVALID), (dict(k=FAKE + 4), ALIGN), (dict(stride=385), ALIGN),
                       (dict(row_stride=132 * 8 + 2), ALIGN), (dict(row=FAKE + 1), ALIGN),
                       (dict(chunk=FAKE + 2), ALIGN), (dict(positions=FAKE + 4), ALIGN), (dict(freq=FAKE + 4), ALIGN),
                       (dict(keys=(ctypes.c_void_p * 3)(FAKE, None, FAKE)), INVALID),
                       (dict(keys=(ctypes.c_void_p * 3)(FAKE, FAKE + 2, FAKE)), ALIGN)]:
        assert call(**kw) == status, kw


def test_bad_norms_are_refused():
    f = fm.lib().fm_add_rmsnorm_fp8

    def call(x=FAKE, xs=256, r=FAKE + 65536, rs=256, gain=None, dtype=0, T=2, H=256, eps=1e-6, group=128,
             out=FAKE + 131072, codes=FAKE, scales=FAKE):
        return f(x, xs, r, rs, gain, dtype, T, H, eps, group, out, codes, scales, None)

    for kw, status in [(dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
                       (dict(dtype=4), INVALID), (dict(T=0), INVALID), (dict(H=0), INVALID), (dict(H=200), UNSUP),
                       (dict(H=32896, xs=32896, rs=32896), UNSUP), (dict(group=64), UNSUP), (dict(eps=-1.0), INVALID),
                       (dict(eps=float("nan")), INVALID), (dict(xs=255), INVALID), (dict(rs=128), INVALID),
                       (dict(out=FAKE, xs=512), INVALID), (dict(out=FAKE + 65536, rs=512), INVALID),
                       (dict(x=FAKE + 4), ALIGN), (dict(r=FAKE + 4), ALIGN), (dict(gain=FAKE + 2), ALIGN),
                       (dict(codes=FAKE + 4), ALIGN), (dict(scales=FAKE + 2), ALIGN), (dict(out=FAKE + 4), ALIGN),
                       (dict(xs=257), ALIGN), (dict(rs=257), ALIGN)]:
        assert call(**kw) == status, kw


def test_rope_frequencies_match_the_oracle_and_refuse():
    # two fp64 powers (1 ulp each side) and up to four roundings after them
    tol = dict(rtol=8 * 2.0 ** -52, atol=0)
    np.testing.assert_allclose(fm.fm_rope_frequencies().numpy(), O.yarn_inv_freq(), **tol)
    np.testing.assert_allclose(fm.fm_rope_frequencies(rope_dim=128, rope_base=10000.0).numpy(),
                               O.yarn_inv_freq(rope_dim=128, base=10000.0), **tol)
    for kw in (dict(rope_dim=0), dict(rope_dim=63), dict(rope_dim=130), dict(rope_base=1.0), dict(rope_factor=0.5)):
        with pytest.raises(fm.FMError) as e:
            fm.fm_rope_frequencies(**kw)
        assert e.value.status == INVALID
    with pytest.raises(ValueError):
        fm.fm_rope_frequencies(hidden=7)
    assert fm.lib().fm_rope_frequencies(None, FAKE) == INVALID


def test_the_binding_refuses_host_tensors_and_shapes():
    pages = torch.zeros(4, 2, 16 * 68, dtype=torch.uint8)
    table = torch.zeros(1, 2, dtype=torch.int32)
    k = torch.zeros(1, 2, 128)
    seq, pos = torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError):
        fm.fm_kv4_append(k, k, pages, pages, table, seq, pos)  # not CUDA tensors
    with pytest.raises(ValueError):
        fm.fm_kv4_append(k[:, :1], k[:, :1], pages, pages, table, seq, pos)  # not the cache's heads
    with pytest.raises(ValueError):
        fm.fm_kv4_append(k, k, pages[..., :100], pages[..., :100], table, seq, pos)
    with pytest.raises(ValueError):
        fm.fm_kv4_append(k, k, pages, pages, table, seq.long(), pos)
    lens = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fm.fm_kv4_attention(k, pages, pages, table, lens)
    cuda_free = [k, pages, pages, table, lens]
    for kw in (dict(window=1 << 32), dict(max_len=-(1 << 33)), dict(window=(1 << 32) + 5)):
        with pytest.raises(ValueError, match="32 bits"):  # a number that 32 bits would cut to another
            fm.fm_kv4_attention(*cuda_free, **kw)
    with pytest.raises(ValueError):
        fm.fm_kv4_attention(k.double(), pages, pages, table, lens)
    with pytest.raises(ValueError):
        fm.fm_kv4_attention(k, pages, pages, table, lens, idx=torch.zeros(1, 3, dtype=torch.int32))  # no count
    with pytest.raises(ValueError):
        fm.fm_kv4_attention(k.expand(2, 2, 128), pages, pages, table, lens)  # another number of rows
    with pytest.raises(ValueError):
        fm.fm_add_rmsnorm_fp8(torch.zeros(2, 256), group=100)
    with pytest.raises(ValueError):
        fm.fm_add_rmsnorm_fp8(torch.zeros(2, 256))
    with pytest.raises(ValueError):
        fm.fm_index_append(k, [torch.zeros(1, 4, 132, dtype=torch.uint8)], seq, seq)  # a key too many


# ----------------------------------------------------------------- oracle pins


def test_oracle_e2m1_and_e8m0_points():
    assert OC.e2m1(np.arange(8)).tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert OC.e2m1(np.arange(8, 16)).tolist() == [0, -0.5, -1, -1.5, -2, -3, -4, -6]
    assert OC.e8m0(np.array([127, 128, 1])).tolist() == [1.0, 2.0, 2.0 ** -126]
    assert np.isnan(OC.e8m0(np.array([255]))[0])


def test_oracle_quantisation_by_hand():
    x = np.zeros((1, 128))
    x[0, :10] = [6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.2, -5.01]  # scale 1: every border, ties to even
    x[0, 32] = 12.0   # exactly 6 * 2
    x[0, 64] = 12.01  # just over
    x[0, 96] = np.inf
    codes, scales = OC.quant4(x)
    assert scales[0].tolist() == [127, 128, 129, 255]
    v = OC.dequant4(codes, scales)[0]
    assert v[:10].tolist() == [6, 4, 4, 2, 2, 1, 1, 0, 0, -6]
    assert v[32] == 12.0 and v[64] == 12.0 and np.isnan(v[96:]).all()
    z, s = OC.quant4(np.zeros((1, 128)))
    assert not z.any() and not s.any()


def test_oracle_quantisation_is_within_half_a_step():
    x = np.random.default_rng(1).standard_normal((50, 128)) * np.exp2(np.arange(50) - 25.0)[:, None]
    codes, scales = OC.quant4(x)
    v = OC.dequant4(codes, scales)
    step = np.repeat(OC.e8m0(scales), 32, axis=1)
    mag = np.abs(x) / step
    half = np.where(mag < 2, 0.25, np.where(mag < 4, 0.5, 1.0)) * step
    assert (np.abs(v - x) <= half).all()
    assert (mag.reshape(50, 4, 32).max(-1) > 3).all()  # the scale is the least that fits


def test_oracle_attention_reduces_to_plain_cases():
    r = np.random.default_rng(2)
    k, v = r.standard_normal((1, 1, 5, 128)), r.standard_normal((1, 1, 5, 128))
    there = np.ones((1, 5), bool)
    zero = np.zeros((1, 1, 1, 128))
    o, *_ = OC.attention(zero, k, v, there, [5])
    np.testing.assert_allclose(o[0, 0, 0], v[0, 0].mean(0))
    o, *_ = OC.attention(zero, k, v, there, [5], window=2)
    np.testing.assert_allclose(o[0, 0, 0], v[0, 0, 3:].mean(0))
    o, *_ = OC.attention(zero, k, v, there, [5], idx=np.array([[4, 9, -1, 0]]), count=[4])
    np.testing.assert_allclose(o[0, 0, 0], (v[0, 0, 4] + v[0, 0, 0]) / 2)
    o, *_ = OC.attention(zero, k, v, there, [5], slopes=[1000.0])
    np.testing.assert_allclose(o[0, 0, 0], v[0, 0, 4])
    o, *_ = OC.attention(np.zeros((1, 3, 1, 128)), k, v, there, [2])
    assert not o[0, 0].any()  # the first of three queries stands before the row's start
    np.testing.assert_allclose(o[0, 1, 0], v[0, 0, 0])


@pytest.mark.parametrize("max_len,max_sel,kw", [
    (16384, 0, {}), (16384, 4096, {}), (300, 0, {}), (300, 4096, {}), (16384, 100, dict(Tq=4)),
    (16384, 16384, dict(n_q_heads=128))])
def test_one_workspace_does_for_every_window_and_list_of_the_same_sizes(max_len, max_sel, kw):
    """Sized once from B, Tq, the heads, max_len and max_sel: a sliding-window layer's buffer also does for a layer
    without a window, and with or without a list (each at the sizes that it was asked for)."""
    c = cache(max_pages=1024, page_table_stride=1024)
    size = fm.lib().fm_kv4_attention_workspace_bytes
    need = set()
    for window in (0, 1, 128, 385, 4096, 1 << 30):
        for listed in ([False, True] if max_sel else [False]):
            d = attn_desc(max_len=max_len, max_sel=max_sel, window=window, idx=FAKE if listed else None,
                          count=FAKE if listed else None, **kw)
            need.add(size(ctypes.byref(c), ctypes.byref(d)))
            # one byte less is refused (before anything is launched)
            assert fm.lib().fm_kv4_attention(ctypes.byref(c), ctypes.byref(d), FAKE, max(need) - 1, None) == INVALID
    assert len(need) == 1 and need.pop() > 0


def test_records_that_would_be_written_over_one_another_are_refused():
    """Keys and values in one pool, or two layers' records in one tensor: the calls would write both to one place."""
    one = cache()
    other = cache(v_pages=FAKE + (1 << 20))
    a = append_desc()
    assert fm.lib().fm_kv4_append(ctypes.byref(one), ctypes.byref(a), None) == INVALID
    a = append_desc(k_hat=FAKE, v_hat=FAKE)
    assert fm.lib().fm_kv4_append(ctypes.byref(other), ctypes.byref(a), None) == INVALID
    f = fm.lib().fm_index_append
    for keys in ((FAKE, FAKE + 4096, FAKE), (FAKE, FAKE, FAKE + 4096)):
        arr = (ctypes.c_void_p * 3)(*keys)
        assert f(FAKE, 0, 384, 5, 3, FAKE, FAKE, FAKE, FAKE, 64, 1, arr, 132 * 8, 2, 8, None) == INVALID
    # reading keys and values from one pool is the caller's choice
    d = attn_desc()
    size = fm.lib().fm_kv4_attention_workspace_bytes
    assert size(ctypes.byref(one), ctypes.byref(d)) == size(ctypes.byref(other), ctypes.byref(d)) > 0


def test_a_list_longer_than_32_bits_is_refused():
    """(Tensors without memory: the check comes before anything looks at their device.)"""
    meta = dict(device="meta")
    q = torch.empty(1, 1, 128, **meta)
    pages, table = torch.empty(1, 1, 16 * 68, dtype=torch.uint8, **meta), torch.empty(1, 1, dtype=torch.int32, **meta)
    one = torch.empty(1, dtype=torch.int32, **meta)
    idx = torch.empty(1, (1 << 32) + 5, dtype=torch.int32, **meta)
    with pytest.raises(ValueError, match="32 bits"):
        fm.fm_kv4_attention(q, pages, pages, table, one, idx=idx, count=one)
    keys = [torch.empty(1, 8, 132, dtype=torch.uint8, **meta)]
    with pytest.raises(ValueError, match="32 bits"):
        fm.fm_index_append(q, keys, one, one, N=5 - (1 << 32))
