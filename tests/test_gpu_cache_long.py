"""The attention over the 4-bit cache where a CTA's share is tens of blocks, so
that its ring of stages goes round many times: every shape of the kernel, over
whole rows, over lists, and over rows whose pages are missing in between.

The reference is the definition in 64 bits on the GPU (elementary operations);
it is compared with the host oracle on a small case first.  Tolerances are
those of test_gpu_cache.py."""
import numpy as np
import pytest
import torch

import oracle.cache as OC

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from learned_kv_chunk_b200 import fm  # noqa: E402  (loads libfm.so; raises if missing)

DEV = torch.device("cuda", 0)
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def values(pages, table, page, head):
    """One kv head of the pages [n] -> [n * page, 128] fp64."""
    blk = pages[table, head]
    codes = blk[:, :page * 64].reshape(-1, page, 64).long()
    scales = blk[:, page * 64:].reshape(-1, page, 4).double()
    n = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(-1, page, 128)
    e, m = (n >> 1) & 3, (n & 1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
    x = torch.where(n >= 8, -mag, mag) * torch.exp2(scales - 127).repeat_interleave(32, dim=-1)
    return x.reshape(-1, 128)


def plain64(q, kp, vp, table, lens, page, idx=None, count=None, window=0, scale=128 ** -0.5):
    """(out, tolerance's parts err_x, abs_v, top_v), each [B, Tq, Hq, 128 or 1] fp64."""
    B, Tq, Hq, _ = q.shape
    Hkv = kp.shape[1]
    G = Hq // Hkv
    out, abs_v = (torch.zeros(B, Tq, Hq, 128, device=DEV, dtype=torch.float64) for _ in range(2))
    err_x, top_v = (torch.zeros(B, Tq, Hq, 1, device=DEV, dtype=torch.float64) for _ in range(2))
    for b in range(B):
        there = (table[b] >= 0) & (table[b] < kp.shape[0])
        at = torch.arange(int(lens[b]), device=DEV) if idx is None else idx[b, :int(count[b])].long()
        at = at[(at >= 0) & (at < int(lens[b]))]
        at = at[there[at // page]]
        for h in range(Hkv):
            k = values(kp, table[b].clamp(0, kp.shape[0] - 1).long(), page, h)[at]
            v = values(vp, table[b].clamp(0, vp.shape[0] - 1).long(), page, h)[at]
            for t in range(Tq):
                p = int(lens[b]) - Tq + t
                ok = at <= p
                if window:
                    ok &= p - at < window
                if not bool(ok.any()):
                    continue
                g = slice(h * G, (h + 1) * G)
                qd, kk, vv = q[b, t, g].double(), k[ok], v[ok]
                x = scale * qd @ kk.T
                w = torch.softmax(x, dim=1)
                out[b, t, g] = w @ vv
                abs_v[b, t, g] = w @ vv.abs()
                e = scale * (qd.abs() @ kk.abs().T + qd.abs().sum(1, keepdim=True) * kk.abs().amax(1) / 16) + x.abs()
                err_x[b, t, g] = e.amax(1, keepdim=True)
                pv = w * vv.abs().amax(1)
                top_v[b, t, g] = 2.0 ** -33 * 12 * kk.shape[0] * pv.amax(1, keepdim=True) + 2.0 ** -24 * pv.sum(1, keepdim=True)
    return out, err_x, abs_v, top_v


def tolerance(dtype, n, out, err_x, abs_v, top_v):
    w = (2.0 ** -20 if dtype == torch.float32 else 2.0 ** -11) + 2.0 ** -23 * (n / 16 + 16)
    half = torch.finfo(dtype).eps / 2
    return (2 * 2.0 ** -20 * err_x + w) * abs_v + top_v + half * out.abs() + torch.finfo(dtype).tiny * half + 1e-37


def make(seed, lens, Hkv, page):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B, per = len(lens), -(-max(lens) // page)
    n = B * per + 2

    def pool():
        p = torch.randint(0, 256, (n, Hkv, page * 68), generator=g, device=DEV, dtype=torch.uint8)
        p[:, :, page * 64:] = torch.randint(121, 128, (n, Hkv, page * 4), generator=g, device=DEV, dtype=torch.uint8)
        return p

    table = torch.randperm(n, generator=g, device=DEV)[:B * per].to(torch.int32).view(B, per)
    return g, pool(), pool(), table


def check(seed, lens, Hq, Hkv, dtype, page=64, Tq=1, table_edit=None, listed=False, **kw):
    g, kp, vp, table = make(seed, lens, Hkv, page)
    if table_edit is not None:
        table_edit(table, kp.shape[0], g)
    q = torch.randn(len(lens), Tq, Hq, 128, generator=g, device=DEV).to(TYPES[dtype])
    n = max(lens)
    if listed:  # a row's positions in no order, every third of them left out
        idx = torch.stack([torch.randperm(n, generator=g, device=DEV) for _ in lens]).to(torch.int32)
        kw.update(idx=idx[:, :n - n // 3].contiguous(), count=torch.full((len(lens),), n - n // 3, device=DEV, dtype=torch.int32))
    kv_len = torch.tensor(lens, device=DEV, dtype=torch.int32)
    o = fm.fm_kv4_attention(q, kp, vp, table, kv_len, **kw)
    again = fm.fm_kv4_attention(q, kp, vp, table, kv_len, **kw)
    out, *parts = plain64(q, kp, vp, table, lens, page, **kw)
    off = (o.double() - out).abs()
    assert torch.equal(o, again)
    assert bool((off <= tolerance(TYPES[dtype], n, out, *parts)).all()), off.max()


SHAPES = [(8, 1, "bf16"), (1, 1, "fp16"), (12, 1, "bf16"), (4, 1, "fp32"), (16, 1, "fp32"), (2, 4, "bf16"), (6, 3, "fp16")]


def test_the_reference_is_the_oracle():
    lens = [70, 33]
    g, kp, vp, table = make(1, lens, 2, 16)
    table[0, 2] = -1
    q = torch.randn(2, 3, 4, 128, generator=g, device=DEV)
    k, there = OC.read_cache(kp.cpu().numpy(), table.cpu().numpy(), 16)
    v, _ = OC.read_cache(vp.cpu().numpy(), table.cpu().numpy(), 16)
    want = OC.attention(q.double().cpu().numpy(), k, v, there, lens, window=40)
    for a, b in zip(want, plain64(q, kp, vp, table, lens, 16, window=40)):
        np.testing.assert_allclose(a, b.cpu().numpy(), rtol=1e-10, atol=1e-14)


@pytest.mark.parametrize("G,Tq,dtype", SHAPES)
@pytest.mark.parametrize("listed", [False, True])
def test_shares_of_tens_of_blocks(G, Tq, dtype, listed):
    """Four rows of up to 40000 tokens and eight kv heads: 34 blocks for a CTA."""
    check(2, [40000, 39999, 40000, 38000], 8 * G, 8, dtype, Tq=Tq, listed=listed)


@pytest.mark.parametrize("G,Tq,dtype", SHAPES)
@pytest.mark.parametrize("page", [16, 48, 128])
def test_the_middle_of_a_row_is_missing(G, Tq, dtype, page):
    """The first pages kept, the middle dropped, the newest kept, at several places; and rows of scattered pages."""
    def edit(table, n_pages, g):
        per = table.shape[1]
        table[0, 384 // page:per - 1000 // page] = -1
        table[1, 2000 // page:per - 3000 // page] = n_pages
        # runs of 1 to 6 blocks of 128 tokens, every other one gone
        at, on = 0, True
        while at < per * page:
            n = 128 * int(torch.randint(1, 7, (1,), generator=g, device=DEV))
            if not on:
                table[2, -(-at // page):(at + n) // page] = -1
            at, on = at + n, not on
        table[3, torch.rand(per, generator=g, device=DEV) < 0.5] = -7
    check(3, [30000, 29000, 30000, 25001], 8 * G, 8, dtype, page=page, Tq=Tq, table_edit=edit)


@pytest.mark.parametrize("G,dtype", [(8, "bf16"), (12, "fp16"), (4, "fp32")])
def test_short_rows_with_a_missing_middle(G, dtype):
    """A few thousand tokens, one kv head, few CTAs with several blocks each."""
    for tokens in (900, 2048, 5000):
        def edit(table, n_pages, g):
            table[:, 24:-8] = -1
        check(4, [tokens, tokens - 1], G, 1, dtype, page=16, table_edit=edit)
    def edit_many(table, n_pages, g):
        table[torch.rand(table.shape, generator=g, device=DEV) < 0.6] = -1
    check(5, [3000] * 300, G, 1, dtype, page=16, table_edit=edit_many)


def test_a_window_over_long_rows_and_pages_missing_in_it():
    def edit(table, n_pages, g):
        table[:, -100:-40] = -1
    check(6, [40000] * 8, 64, 8, "bf16", window=20000, table_edit=edit)
    check(6, [40000] * 8, 96, 8, "bf16", window=20000, table_edit=edit)


@pytest.mark.parametrize("B,n,G,dtype", [(40, 900, 8, "bf16"), (300, 700, 12, "fp32"), (3000, 60, 2, "bf16"),
                                         (3000, 60, 24, "fp16")])
@pytest.mark.parametrize("listed", [False, True])
def test_more_rows_than_lanes(B, n, G, dtype, listed):
    """Their places among the CTAs come from the block's scan: rows of every length, with lists and without."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, n + 1, B)]
    lens[0] = n
    check(7, lens, G, 1, dtype, page=16, listed=listed)


@pytest.mark.parametrize("Tq", [1, 5])
def test_as_many_heads_as_there_may_be(Tq):
    check(8, [50, 200], 1024, 1024, "bf16", page=16, Tq=Tq)
    check(8, [50, 700], 1024, 1, "fp32", page=16, Tq=Tq)
