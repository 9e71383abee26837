"""The operators around the 4-bit paged cache, as cases that can be timed and compared.

Four operators of a decode step that stand next to the retriever: the append
of keys and values to a paged cache held in 4 bits (with the position
rotation on the way), the attention over that cache, the append of indexer
keys as the 132-byte records that the retriever scores, and the residual
addition with RMSNorm and an e4m3 output with scales.

`run` computes each in its plain form (elementary torch operations) or, where
`own` is true, by the library's calls.

The 4-bit record of a token and head: 128 e2m1 codes (two to a byte, the
even dimension in the low half) and four e8m0 scale bytes, one for each 32
dimensions.  A (page, head) block holds the codes of its page_size tokens
(64 bytes each), then their scales (4 bytes each).
"""
import math

import torch

own = False

D = 128
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZES = {"fp32": 4, "bf16": 2, "fp16": 2}


# ------------------------------------------------------------------ the cases


def _attn(name, B, Tq, Hq, Hkv, cap, dtype, page=64, ragged=False, softcap=0.0, slopes=False, window=0,
          start=False, sel=0):
    c = dict(op="attention", B=B, Tq=Tq, Hq=Hq, Hkv=Hkv, cap=cap, dtype=dtype, page=page, ragged=ragged,
             softcap=softcap, slopes=slopes, window=window, start=start, sel=sel)
    return dict(c, name=name) if name else c


def _append(name, T, B, Hq, Hkv, cap, dtype, page=64, rope_dim=64, prompt=False):
    c = dict(op="append", T=T, B=B, Hq=Hq, Hkv=Hkv, cap=cap, dtype=dtype, page=page, rope_dim=rope_dim,
             prompt=prompt)
    return dict(c, name=name) if name else c


def _index(name, T, B, L, N, dtype):
    c = dict(op="index", T=T, B=B, L=L, N=N, dtype=dtype)
    return dict(c, name=name) if name else c


def _norm(name, T, H, dtype, group=128):
    c = dict(op="norm", T=T, H=H, dtype=dtype, group=group)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user, a short conversation of odd length: latency counts
        _attn("attention 1 row x 1001", 1, 1, 32, 8, 1001, "bf16", page=16),
        # a serving batch of ragged lengths, capped scores
        _attn("attention 32 ragged x 8192", 32, 1, 64, 8, 8192, "bf16", ragged=True, softcap=30.0),
        # long contexts: the cache's bytes count
        _attn("attention 8 x 131072", 8, 1, 64, 8, 131072, "bf16"),
        # the retriever's kept tokens only, 32 heads over one memory (the decode loop's layout), fp32
        _attn("attention kept 4096 of 65536", 8, 1, 32, 1, 65536, "fp32", sel=4096),
        # drafts of four tokens with a distance bias, a sliding window and document starts
        _attn("attention drafts 16 x 16384", 16, 4, 32, 4, 16384, "fp16", ragged=True, slopes=True,
              window=4096, start=True),
        # one decode step of 64 rows: keys, values and queries rotated, keys and values stored
        _append("append 64 tokens", 64, 64, 64, 8, 65536, "bf16"),
        # a prefill batch: ragged prompts, padded at the end
        _append("append prompts of 8192", 8192, 5, 32, 8, 16384, "fp16", page=16, rope_dim=128, prompt=True),
        # one step's new indexer keys of the three layers
        _index("index 64 chunks", 64, 64, 3, 4096, "fp32"),
        # a prompt's indexer keys
        _index("index 32768 chunks", 32768, 4, 3, 16384, "bf16"),
        # the hidden state of a decode step (the retriever's hidden size)
        _norm("norm 64 x 4096", 64, 4096, "fp32"),
        # a prefill batch, one scale for each row
        _norm("norm 16384 x 8192", 16384, 8192, "bf16", group=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "index", "norm"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op == "attention":
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 32])
        Tq = rng.choice([1, 1, 1, 2, 3, 5, 8])
        cap = _log(rng, 1, 131072)
        B = min(_log(rng, 1, 64), max(1, 8 * 131072 * 8 // (cap * Hkv * max(1, G * Tq // 8))))
        sel = rng.choice([0, 0, _log(rng, 1, 4096)])
        return _attn(None, B, Tq, Hkv * G, Hkv, cap, dtype, page=rng.choice([16, 32, 48, 64, 128]),
                     ragged=rng.random() < 0.6, softcap=rng.choice([0.0, 0.0, 20.0, 50.0]),
                     slopes=rng.random() < 0.3, window=rng.choice([0, 0, _log(rng, 1, 8192)]),
                     start=rng.random() < 0.3, sel=sel)
    if op == "append":
        prompt = rng.random() < 0.5
        T = _log(rng, 2, 8192) if prompt else _log(rng, 1, 256)
        return _append(None, T, _log(rng, 1, 8) if prompt else T, rng.choice([0, 8, 32, 64]),
                       rng.choice([1, 2, 4, 8]), _log(rng, 64, 65536), dtype, page=rng.choice([16, 32, 48, 64]),
                       rope_dim=rng.choice([0, 64, 128]), prompt=prompt)
    if op == "index":
        T = _log(rng, 1, 32768)
        B = rng.choice([1, 3, 4, 8])
        return _index(None, T, B, rng.choice([1, 2, 3, 4]), (T // B + 8 + _log(rng, 1, 4096)) // 4 * 4, dtype)
    H = 128 * _log(rng, 1, 128)
    return _norm(None, _log(rng, 1, 16384 * 8192 // max(H, 8192)), H, dtype, group=rng.choice([128, H]))


# ------------------------------------------------------------- what is in hand


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _freqs(rope_dim):
    """Rotary frequencies with YaRN's interpolation (base 160000, factor 16, 65536 positions, 32 and 1 turns)."""
    def dim_of(turns):
        return rope_dim * math.log(65536.0 / (turns * 2.0 * math.pi)) / (2.0 * math.log(160000.0))
    lo, hi = max(math.floor(dim_of(32.0)), 0), min(math.ceil(dim_of(1.0)), rope_dim - 1)
    j = torch.arange(rope_dim // 2, dtype=torch.float64)
    inv = 160000.0 ** (-2.0 * j / rope_dim)
    ramp = ((j - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
    return (inv * (1.0 - ramp) + inv / 16.0 * ramp).cuda()


def _lengths(c, cpu):
    if not c["ragged"]:
        return torch.full((c["B"],), c["cap"], dtype=torch.int32)
    n = torch.randint(0, c["cap"] + 1, (c["B"],), generator=cpu, dtype=torch.int32)
    n[-1] = c["cap"]
    if c["B"] > 3:
        n[0] = 0  # a row that holds nothing yet
    return n


def _prepare_attention(c, seed):
    g, cpu = _gen(seed), torch.Generator().manual_seed(int(seed))
    B, Hkv, page = c["B"], c["Hkv"], c["page"]
    per = -(-c["cap"] // page)
    n_pages = B * per + 3
    lens = _lengths(c, cpu)
    s = dict(c=c, kv_len=lens.cuda())
    # pages of all rows in one pool, in no order
    order = torch.randperm(n_pages, generator=g, device="cuda")[: B * per].to(torch.int32).view(B, per)
    used = (s["kv_len"].view(B, 1) + page - 1) // page
    s["page_table"] = torch.where(torch.arange(per, device="cuda").view(1, per) < used, order, -1).to(torch.int32)
    for name in ("k_pages", "v_pages"):
        p = torch.randint(0, 256, (n_pages, Hkv, page * 68), generator=g, device="cuda", dtype=torch.uint8)
        p[:, :, page * 64:] = torch.randint(123, 127, (n_pages, Hkv, page * 4), generator=g, device="cuda",
                                            dtype=torch.uint8)
        s[name] = p
    s["q"] = (1.5 * torch.randn(B, c["Tq"], c["Hq"], D, generator=g, device="cuda")).to(DTYPES[c["dtype"]])
    s["slopes"] = (torch.exp2(-8.0 * (torch.arange(c["Hq"], device="cuda") + 1) / c["Hq"]).float()
                   if c["slopes"] else None)
    s["kv_start"] = ((torch.rand(B, generator=cpu) * 0.2 * lens).to(torch.int32).cuda() if c["start"] else None)
    s["idx"] = s["count"] = None
    if c["sel"]:
        # the kept positions of each row, ascending: a random subset of what the row holds
        sel = c["sel"]
        score = torch.rand(B, c["cap"], generator=g, device="cuda")
        score.masked_fill_(torch.arange(c["cap"], device="cuda").view(1, -1) >= s["kv_len"].view(B, 1), -1.0)
        k = min(sel, c["cap"])
        top = torch.topk(score, k, dim=1).indices
        s["count"] = torch.minimum(s["kv_len"], torch.tensor(k, device="cuda")).to(torch.int32)
        none = torch.arange(k, device="cuda").view(1, -1) >= s["count"].view(B, 1)
        top = torch.sort(top.masked_fill(none, 1 << 40), dim=1).values
        s["idx"] = torch.full((B, sel), -1, device="cuda", dtype=torch.int32)
        s["idx"][:, :k] = torch.where(none, -1, top).to(torch.int32)
    return s


def _prepare_append(c, seed):
    g, cpu = _gen(seed), torch.Generator().manual_seed(int(seed))
    T, B, Hq, Hkv, page = c["T"], c["B"], c["Hq"], c["Hkv"], c["page"]
    dt = DTYPES[c["dtype"]]
    # the projections' output: queries, keys and values of a token side by side
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(dt)
    heads = qkv.view(T, Hq + 2 * Hkv, D)
    if c["prompt"]:  # ragged prompts, one after the other, then padding
        live = max(1, T - T // 50)
        cuts = torch.sort(torch.randint(0, live + 1, (B - 1,), generator=cpu)).values.tolist()
        n = [b - a for a, b in zip([0] + cuts, cuts + [live])]
        first = torch.randint(0, c["cap"] + 1, (B,), generator=cpu).tolist()
    else:  # a token of every row
        n, first = [1] * B, torch.randint(0, c["cap"], (B,), generator=cpu).tolist()
    seq = torch.full((T,), -1, dtype=torch.int32)
    pos = torch.full((T,), -1, dtype=torch.int64)
    at = 0
    for b in range(B):
        seq[at:at + n[b]] = b
        pos[at:at + n[b]] = first[b] + torch.arange(n[b])
        at += n[b]
    lo = [f // page for f in first]
    need = [(first[b] + n[b] + page - 1) // page - lo[b] for b in range(B)]
    n_pages = sum(need) + 2
    table = torch.full((B, max(lo[b] + need[b] for b in range(B)) + 1), -1, dtype=torch.int32)
    order = torch.randperm(n_pages, generator=cpu).to(torch.int32)
    at = 0
    for b in range(B):  # the pages before the new tokens lie elsewhere: only those that are written are here
        table[b, lo[b]:lo[b] + need[b]] = order[at:at + need[b]]
        at += need[b]
    return dict(c=c, q=heads[:, :Hq], k=heads[:, Hq:Hq + Hkv], v=heads[:, Hq + Hkv:], seq=seq.cuda(),
                pos=pos.cuda(), page_table=table.cuda(), live=torch.nonzero(seq >= 0).view(-1).cuda(),
                inv_freq=_freqs(c["rope_dim"]) if c["rope_dim"] else None,
                k_pages=torch.zeros(n_pages, Hkv, page * 68, device="cuda", dtype=torch.uint8),
                v_pages=torch.zeros(n_pages, Hkv, page * 68, device="cuda", dtype=torch.uint8),
                q_out=torch.zeros(T, Hq, D, device="cuda", dtype=dt) if Hq else None,
                k_hat=torch.zeros(T, Hkv, D, device="cuda", dtype=torch.bfloat16),
                v_hat=torch.zeros(T, Hkv, D, device="cuda", dtype=torch.bfloat16))


def _prepare_index(c, seed):
    g = _gen(seed)
    T, B, L, N = c["T"], c["B"], c["L"], c["N"]
    t = torch.arange(T, device="cuda")
    row = (t % B).to(torch.int32)  # row b gets the tokens t with t % B == b, from a chunk of its own on
    first = torch.randint(0, N - -(-T // B) + 1, (B,), generator=g, device="cuda")
    chunk = (first[t % B] + t // B).to(torch.int32)
    return dict(c=c, k=torch.randn(T, L, D, generator=g, device="cuda").to(DTYPES[c["dtype"]]), row=row, chunk=chunk,
                positions=4 * chunk.long(), inv_freq=_freqs(64),
                comp_k=[torch.zeros(B, N, 132, device="cuda", dtype=torch.uint8) for _ in range(L)])


def _prepare_norm(c, seed):
    g = _gen(seed)
    dt = DTYPES[c["dtype"]]
    x = torch.randn(c["T"], c["H"], generator=g, device="cuda")
    r = 2.0 * torch.randn(c["T"], c["H"], generator=g, device="cuda")
    return dict(c=c, x=x.to(dt), residual=r.to(dt),
                gain=(1.0 + 0.02 * torch.randn(c["H"], generator=g, device="cuda")).to(dt))


def prepare(case, seed):
    return {"attention": _prepare_attention, "append": _prepare_append, "index": _prepare_index,
            "norm": _prepare_norm}[case["op"]](case, seed)


# ------------------------------------------------------------ the plain forms

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pairs(device):
    """The two values of every code byte: [256, 2] fp32."""
    v = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=device)
    b = torch.arange(256, device=device)
    return torch.stack([v[b & 15], v[b >> 4]], dim=1)


def _dequant(codes, scales):
    """codes [..., 64] and scales [..., 4] (bytes) -> fp32 [..., 128]."""
    x = _pairs(codes.device)[codes.int()].reshape(*codes.shape[:-1], 4, 32)
    return (x * torch.exp2(scales.float() - 127.0).unsqueeze(-1)).reshape(*codes.shape[:-1], D)


def _plain_attention(s):
    c = s["c"]
    B, Tq, Hq, Hkv, page = c["B"], c["Tq"], c["Hq"], c["Hkv"], c["page"]
    G = Hq // Hkv
    dev = s["q"].device

    def memory(pages):
        if s["idx"] is not None:  # [B, sel, Hkv, ...] of the kept tokens
            at = s["idx"].clamp(min=0).long()
            p = torch.gather(s["page_table"], 1, at // page).clamp(min=0).long()
            block = pages[:, :, : page * 64].unflatten(2, (page, 64))
            scale = pages[:, :, page * 64:].unflatten(2, (page, 4))
            x = _dequant(block[p, :, at % page], scale[p, :, at % page])
            return x.transpose(1, 2)  # [B, Hkv, sel, D]
        block = pages[s["page_table"].clamp(min=0).long()]  # [B, per, Hkv, page * 68]
        x = _dequant(block[..., : page * 64].unflatten(-1, (page, 64)),
                     block[..., page * 64:].unflatten(-1, (page, 4)))
        return x.transpose(1, 2).reshape(B, Hkv, -1, D)

    q = s["q"].float().view(B, Tq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Tq, D)
    x = torch.matmul(q, memory(s["k_pages"]).transpose(2, 3)) * D ** -0.5
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    n = x.shape[-1]
    lens = s["kv_len"].long().view(B, 1, 1)
    t = lens - Tq + torch.arange(Tq, device=dev).view(1, Tq, 1)  # the queries' positions
    if s["idx"] is not None:
        j = s["idx"].long().view(B, 1, n)
        seen = (j >= 0) & (torch.arange(n, device=dev).view(1, 1, n) < s["count"].view(B, 1, 1))
    else:
        j = torch.arange(n, device=dev).view(1, 1, n)
        seen = j >= 0
    seen = seen & (j <= t)
    if c["window"]:
        seen = seen & (t - j < c["window"])
    if s["kv_start"] is not None:
        seen = seen & (j >= s["kv_start"].view(B, 1, 1))
    x = x.view(B, Hkv, G, Tq, n)
    if s["slopes"] is not None:
        x = x + s["slopes"].view(1, Hkv, G, 1, 1) * (j - t).float().view(B, 1, 1, Tq, n)
    x = x.masked_fill(~seen.view(B, 1, 1, Tq, n), float("-inf"))
    m = x.amax(dim=-1, keepdim=True)
    e = torch.exp(x - torch.where(m == float("-inf"), 0.0, m))
    total = e.sum(dim=-1, keepdim=True)
    p = e / torch.where(total == 0.0, 1.0, total)
    o = torch.matmul(p.view(B, Hkv, G * Tq, n), memory(s["v_pages"]))
    o = o.view(B, Hkv, G, Tq, D).permute(0, 3, 1, 2, 4).reshape(B, Tq, Hq, D)
    return o.to(s["q"].dtype)


def _rotate(x, positions, inv_freq):
    """x [T, heads, D] -> fp64, its last 2 * len(inv_freq) dimensions rotated in half-split pairs.  In 64 bits, as
    the codes of values next to a border depend on it; the cosines and sines are rounded to fp32 once."""
    x = x.double()
    if inv_freq is None:
        return x
    half = inv_freq.numel()
    a = positions.double().view(-1, 1, 1) * inv_freq.view(1, 1, half)
    c, s = torch.cos(a).float().double(), torch.sin(a).float().double()
    keep, x1, x2 = x[..., : D - 2 * half], x[..., D - 2 * half: D - half], x[..., D - half:]
    return torch.cat([keep, x1 * c - x2 * s, x2 * c + x1 * s], dim=-1)


def _quant4(x):
    """fp64 [..., 128] -> code bytes [..., 64], scale bytes [..., 4], the values they stand for (bf16)."""
    g = x.reshape(*x.shape[:-1], 4, 32)
    top = g.abs().amax(dim=-1)
    man, exp = torch.frexp(top)
    e = torch.where(man <= 0.75, exp - 3, exp - 2).clamp(-126, 125)  # the least e with top <= 6 * 2^e
    y = g.abs() * torch.exp2(-e.double()).unsqueeze(-1)
    # round to nearest, ties to the even code
    code = ((y > 0.25).int() + (y >= 0.75).int() + (y > 1.25).int() + (y >= 1.75).int() + (y > 2.5).int()
            + (y >= 3.5).int() + (y > 5.0).int())
    neg = (g < 0.0) & (code > 0)
    value = torch.tensor(_E2M1, device=x.device, dtype=torch.float64)[code] * torch.where(neg, -1.0, 1.0)
    value = (value * torch.exp2(e.double()).unsqueeze(-1)).reshape(x.shape).to(torch.bfloat16)
    code = (code + 8 * neg.int()).reshape(*x.shape[:-1], 64, 2)
    scale = torch.where(top > 0.0, e + 127, 0)
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), scale.to(torch.uint8), value


def _plain_append(s):
    c = s["c"]
    page, live = c["page"], s["live"]
    seq, pos = s["seq"][live].long(), s["pos"][live]
    p = s["page_table"][seq, pos // page].long()
    slot = pos % page
    for x, pages, hat, f in ((s["k"], s["k_pages"], s["k_hat"], s["inv_freq"]),
                             (s["v"], s["v_pages"], s["v_hat"], None)):
        codes, scales, value = _quant4(_rotate(x[live], pos, f))
        pages[:, :, : page * 64].unflatten(2, (page, 64))[p, :, slot] = codes
        pages[:, :, page * 64:].unflatten(2, (page, 4))[p, :, slot] = scales
        hat[live] = value
    if c["Hq"]:
        s["q_out"][live] = _rotate(s["q"][live], pos, s["inv_freq"]).to(s["q"].dtype)
    return _append_outputs(s)


def _append_outputs(s):
    """The values that the new records stand for, the rotated queries, and the cache itself."""
    out = dict(k=s["k_hat"], v=s["v_hat"], k_pages=s["k_pages"], v_pages=s["v_pages"])
    if s["c"]["Hq"]:
        out["q"] = s["q_out"]
    return out


def _e4m3(y, scale):
    """fp32 values over their scale (0 where the scale is 0) as e4m3."""
    y = y / torch.where(scale == 0.0, 1.0, scale)
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _plain_index(s):
    x = _rotate(s["k"], s["positions"], s["inv_freq"]).float()
    T, L = x.shape[:2]
    for step in (1, 2, 4, 8, 16, 32, 64):  # the Walsh-Hadamard butterflies
        x = x.view(T, L, -1, 2, step)
        x = torch.stack([x[:, :, :, 0] + x[:, :, :, 1], x[:, :, :, 0] - x[:, :, :, 1]], dim=3)
    x = x.view(T, L, D) * (128.0 ** -0.5)
    scale = x.abs().amax(dim=-1, keepdim=True) / 448.0
    rec = torch.cat([_e4m3(x, scale).view(torch.uint8), scale.view(torch.uint8)], dim=-1)
    row, chunk = s["row"].long(), s["chunk"].long()
    for l, keys in enumerate(s["comp_k"]):
        keys[row, chunk] = rec[:, l]
    return _index_outputs(s)


def _index_outputs(s):
    """The records of every row: their codes as the e4m3 values they are, and their scales."""
    return [dict(codes=k[..., :D].view(torch.float8_e4m3fn), scale=k[..., D:].view(torch.float32))
            for k in s["comp_k"]]


def _plain_norm(s):
    c = s["c"]
    z = s["x"].float() + s["residual"].float()
    y = z * torch.rsqrt((z * z).mean(dim=-1, keepdim=True) + 1e-6) * s["gain"].float()
    y = y.view(c["T"], -1, c["group"])
    scale = y.abs().amax(dim=-1, keepdim=True) / 448.0
    return dict(sum=z.to(s["x"].dtype), codes=_e4m3(y, scale).view(c["T"], c["H"]), scale=scale.squeeze(-1))


def run(s):
    op = s["c"]["op"]
    if not own:
        return {"attention": _plain_attention, "append": _plain_append, "index": _plain_index,
                "norm": _plain_norm}[op](s)
    from learned_kv_chunk_b200 import fm
    c = s["c"]
    if op == "attention":
        return fm.fm_kv4_attention(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["kv_len"],
                                   softcap=c["softcap"], slopes=s["slopes"], window=c["window"],
                                   kv_start=s["kv_start"], idx=s["idx"], count=s["count"])
    if op == "append":
        fm.fm_kv4_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"], s["seq"], s["pos"],
                         inv_freq=s["inv_freq"], q=s["q"] if c["Hq"] else None, q_out=s["q_out"],
                         k_hat=s["k_hat"], v_hat=s["v_hat"])
        return _append_outputs(s)
    if op == "index":
        fm.fm_index_append(s["k"], s["comp_k"], s["row"], s["chunk"], inv_freq=s["inv_freq"],
                           positions=s["positions"])
        return _index_outputs(s)
    total, codes, scale = fm.fm_add_rmsnorm_fp8(s["x"], s["residual"], s["gain"], eps=1e-6, group=c["group"])
    return dict(sum=total, codes=codes, scale=scale)


# ------------------------------------------------------------------ the bounds


def work(case):
    c = case
    es = SIZES[c["dtype"]]
    if c["op"] == "attention":
        tokens = c["cap"] / 2 if c["ragged"] else c["cap"]
        if c["window"]:
            tokens = min(tokens, c["window"] + c["Tq"] - 1)
        if c["sel"]:
            tokens = min(tokens, c["sel"] * (tokens / c["cap"] if c["window"] else 1.0))
        tokens = max(1.0, tokens)
        qo = 2 * c["B"] * c["Tq"] * c["Hq"] * D * es
        return {"bytes": c["B"] * c["Hkv"] * tokens * 136 + qo,
                "flops": 4 * c["B"] * c["Tq"] * c["Hq"] * tokens * D}
    if c["op"] == "append":
        T, Hq, Hkv = c["T"], c["Hq"], c["Hkv"]
        return {"bytes": T * ((2 * Hq + 2 * Hkv) * D * es + 2 * Hkv * (68 + 2 * D) + 12),
                "flops": T * ((Hq + Hkv) * c["rope_dim"] * 3 + 2 * Hkv * D * 3)}
    if c["op"] == "index":
        return {"bytes": c["T"] * (c["L"] * (D * es + 132) + 16), "flops": c["T"] * c["L"] * D * 12}
    return {"bytes": c["T"] * (c["H"] * (3 * es + 1) + 4 * c["H"] // c["group"]) + c["H"] * es,
            "flops": c["T"] * c["H"] * 6}


# ------------------------------------------------------------ in 64 bits, apart


def _values4(codes, scales):
    """Code and scale bytes -> fp64, from the formats' fields: sign, two exponent bits (bias 1), one mantissa bit."""
    n = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).to(torch.int64)
    e, m = (n >> 1) & 3, (n & 1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.pow(2.0, (e - 1).double()))
    grown = torch.pow(2.0, scales.double() - 127).repeat_interleave(32, dim=-1)
    return torch.where(n >= 8, -mag, mag) * grown


def _exact_attention(c, seed):
    s = _prepare_attention(c, seed)
    B, Tq, Hq, Hkv, page = c["B"], c["Tq"], c["Hq"], c["Hkv"], c["page"]
    G = Hq // Hkv
    out = torch.zeros(B, Tq, Hq, D, device="cuda", dtype=torch.float64)
    lens = s["kv_len"].tolist()
    for b in range(B):
        if s["idx"] is not None:
            at = s["idx"][b, : int(s["count"][b])].long()
        else:
            at = torch.arange(lens[b], device="cuda")
        if s["kv_start"] is not None:
            at = at[at >= s["kv_start"][b]]
        if c["window"]:
            at = at[at > lens[b] - Tq - c["window"]]
        if at.numel() == 0:
            continue
        pg, slot = s["page_table"][b][at // page].long(), at % page
        for h in range(Hkv):
            kc, vc = s["k_pages"][:, h], s["v_pages"][:, h]
            byte = slot.view(-1, 1) * 64 + torch.arange(64, device="cuda")
            sbyte = page * 64 + slot.view(-1, 1) * 4 + torch.arange(4, device="cuda")
            k = _values4(kc[pg.view(-1, 1), byte], kc[pg.view(-1, 1), sbyte])
            v = _values4(vc[pg.view(-1, 1), byte], vc[pg.view(-1, 1), sbyte])
            for t in range(Tq):
                p = lens[b] - Tq + t
                ok = at <= p
                if c["window"]:
                    ok &= p - at < c["window"]
                if not bool(ok.any()):
                    continue
                w = (s["q"][b, t, h * G:(h + 1) * G].double() @ k.T) / math.sqrt(D)
                if c["softcap"]:
                    w = torch.tanh(w / c["softcap"]) * c["softcap"]
                if s["slopes"] is not None:
                    w = w - s["slopes"][h * G:(h + 1) * G].double().view(G, 1) * (p - at).double()
                w[:, ~ok] = float("-inf")
                out[b, t, h * G:(h + 1) * G] = torch.softmax(w, dim=1) @ v
    return out


def _turned(x, positions, inv_freq):
    """fp64 rotation by complex products; cosines and sines of fp64 angles, rounded to fp32 as the operator has them."""
    x = x.double()
    if inv_freq is None:
        return x
    half = inv_freq.numel()
    a = torch.outer(positions.double(), inv_freq).unsqueeze(1)
    w = torch.complex(a.cos().float().double(), a.sin().float().double())
    z = torch.complex(x[..., D - 2 * half: D - half].contiguous(), x[..., D - half:].contiguous()) * w
    return torch.cat([x[..., : D - 2 * half], z.real, z.imag], dim=-1)


def _nearest4(x):
    """fp64 [..., 128] -> the values of its 4-bit form."""
    g = x.unflatten(-1, (4, 32))
    top = g.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top == 0, 1.0, top) / 6.0))
    e = torch.where(top > 6.0 * torch.pow(2.0, e), e + 1, torch.where(top <= 3.0 * torch.pow(2.0, e), e - 1, e))
    y = (g / torch.pow(2.0, e)).abs()
    # steps of 1/2 up to 2, of 1 up to 4, of 2 above; torch.round goes to even
    r = torch.where(y < 2, torch.round(y * 2) / 2, torch.where(y < 4, torch.round(y), torch.round(y / 2) * 2))
    return (torch.sign(g) * r * torch.pow(2.0, e)).flatten(-2)


def _exact_append(c, seed):
    s = _prepare_append(c, seed)
    live = s["seq"] >= 0
    keep = live.view(-1, 1, 1)
    out = dict(k=torch.where(keep, _nearest4(_turned(s["k"], s["pos"], s["inv_freq"])), 0.0),
               v=torch.where(keep, _nearest4(s["v"].double()), 0.0), k_pages=None, v_pages=None)
    if c["Hq"]:
        out["q"] = torch.where(keep, _turned(s["q"], s["pos"], s["inv_freq"]), 0.0)
    return out


def _exact_index(c, seed):
    s = _prepare_index(c, seed)
    i = torch.arange(D)
    sign = torch.tensor([[1.0 if bin(int(a) & int(b)).count("1") % 2 == 0 else -1.0 for b in i] for a in i],
                        dtype=torch.float64, device="cuda")
    x = _turned(s["k"], s["positions"], s["inv_freq"]) @ (sign / math.sqrt(D))
    out = []
    for l in range(c["L"]):
        scale = torch.zeros(c["B"], c["N"], 1, device="cuda", dtype=torch.float64)
        codes = torch.zeros(c["B"], c["N"], D, device="cuda", dtype=torch.float64)
        top = x[:, l].abs().amax(-1, keepdim=True) / 448.0
        scale[s["row"].long(), s["chunk"].long()] = top
        codes[s["row"].long(), s["chunk"].long()] = x[:, l] / top
        out.append(dict(codes=codes, scale=scale))
    return out


def _exact_norm(c, seed):
    s = _prepare_norm(c, seed)
    z = s["x"].double() + s["residual"].double()
    y = z / torch.sqrt(z.pow(2).mean(-1, keepdim=True) + 1e-6) * s["gain"].double()
    g = y.unflatten(-1, (-1, c["group"]))
    top = g.abs().amax(-1, keepdim=True) / 448.0
    return dict(sum=z, codes=(g / top).flatten(-2), scale=top.squeeze(-1))


def exact(case, seed):
    return {"attention": _exact_attention, "append": _exact_append, "index": _exact_index,
            "norm": _exact_norm}[case["op"]](case, seed)
