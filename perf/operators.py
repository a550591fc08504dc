"""The serving operators: what is measured, on which inputs, and their plain forms.

Five operators make one step of a served model: the norm in front of a linear layer with its
8-bit output, the product of a few rows with 4-bit weights, the block tables of a paged cache,
the append to that cache, and the attention that reads it.  A case names its operator in "op".
"""
import math

import numpy as np
import torch

own = False

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the 3 low bits of an E2M1 code


def listed():
    return [
        # sixteen requests, each a token further: the table work of an ordinary decode step
        dict(name="tables_decode", op="tables", B=16, page=64, max_len=4096, max_new=1, pad=0),
        # a full server: decoding requests mixed with prompts being read, small pages, a padded batch
        dict(name="tables_mixed", op="tables", B=509, page=16, max_len=32768, max_new=1024, pad=100),
        # one new token for each of 64 sequences of 8 heads
        dict(name="store_decode", op="store", B=64, H=8, D=128, page=64, max_len=4096, new=1, pad=0),
        # prompts read in one go: ragged, pages that begin and end inside a prompt
        dict(name="store_prefill", op="store", B=7, H=8, D=128, page=16, max_len=500, new=2041, pad=19),
        # one user, a short context, grouped heads: latency counts
        dict(name="attn_one_short", op="attn", B=1, H=8, G=4, D=128, page=16, max_len=1000, new=1, pad=0),
        # 32 ragged sequences of up to 32768 tokens, one new token each: the cache's bytes count
        dict(name="attn_decode_long", op="attn", B=32, H=8, G=4, D=128, page=64, max_len=32768, new=1, pad=0),
        # two prompts read in pieces of up to 2048 tokens behind a context: the products count
        dict(name="attn_extend", op="attn", B=2, H=8, G=4, D=128, page=64, max_len=8191, new=2048, pad=0),
        # one token of a 4096-wide model
        dict(name="norm_token", op="norm", T=1, K=4096, residual=True, hadamard=0),
        # a prompt of 8192 tokens, rotated for rotated weights
        dict(name="norm_prefill", op="norm", T=8192, K=4096, residual=True, hadamard=32),
        # the attention output projection for one token, rotated weights, bf16 activations
        dict(name="matvec_nv_1", op="matvec", fmt="nvfp4", M=1, N=4096, K=4096, x8=False, hadamard=16),
        # the way down of the feed-forward layer, a few tokens
        dict(name="matvec_nv_5", op="matvec", fmt="nvfp4", M=5, N=4096, K=14336, x8=False, hadamard=0),
        # the way up of the feed-forward layer, sixteen tokens in 8 bits from the norm
        dict(name="matvec_mx_16", op="matvec", fmt="mxfp4", M=16, N=14336, K=4096, x8=True, hadamard=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "store", "attn", "attn", "norm", "matvec", "matvec"])
    if op == "tables":
        return dict(op=op, B=_log(rng, 1, 1024), page=rng.choice([16, 32, 64, 128]), max_len=_log(rng, 64, 32768),
                    max_new=_log(rng, 1, 1024), pad=rng.choice([0, rng.randrange(1, 300)]))
    if op == "store":
        new = _log(rng, 1, 2048)
        return dict(op=op, B=_log(rng, 1, max(2, min(256, 16384 // new))), H=_log(rng, 1, 16), D=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64, 128]), max_len=_log(rng, 16, 4096), new=new,
                    pad=rng.choice([0, rng.randrange(1, 100)]))
    if op == "attn":
        D, H, G = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8]), rng.randrange(1, 9)
        page, pad = rng.choice([16, 32, 64, 128]), rng.choice([0, rng.randrange(1, 20)])
        if rng.random() < 0.5:  # decoding: one token, or the few of a draft
            max_len = _log(rng, 16, 32768)
            return dict(op=op, B=_log(rng, 1, max(1, min(64, 500000 // max_len))), H=H, G=G, D=D, page=page,
                        max_len=max_len, new=rng.choice([1, 1, rng.randrange(2, 9)]), pad=pad)
        new = _log(rng, 9, 2000)
        max_len = _log(rng, 16, 6000)
        return dict(op=op, B=_log(rng, 1, max(1, min(8, 2000 // new))), H=H, G=G, D=D, page=page, max_len=max_len,
                    new=new, pad=pad)
    if op == "norm":
        K = 32 * _log(rng, 2, 448)
        return dict(op=op, T=_log(rng, 1, max(1, min(8192, 30000000 // K))), K=K, residual=rng.random() < 0.7,
                    hadamard=rng.choice([0, 16, 32]))
    x8 = rng.random() < 0.5
    fmt = rng.choice(["nvfp4", "mxfp4"])
    return dict(op=op, fmt=fmt, M=rng.randrange(1, 17), N=_log(rng, 64, 14336), K=64 * _log(rng, 1, 224), x8=x8,
                hadamard=0 if x8 else rng.choice([0, 16 if fmt == "nvfp4" else 32]))


# ---------------------------------------------------------------- inputs
def _lengths(case):
    """Tokens held before the call and new tokens, by request: the first at its largest, some without
    a new token in a padded batch, the others ragged.  They belong to the case, whatever the seed."""
    B = case["B"]
    r = np.random.RandomState(B + 1000 * case["max_len"])
    new_top = case["max_new"] if case["op"] == "tables" else case["new"]
    if new_top == 1:
        new = np.ones(B, np.int64)
    else:
        new = r.randint(max(1, new_top // 2), new_top + 1, B)
        if case["op"] == "tables":  # most requests decode, some read a prompt
            new = np.where(r.rand(B) < 0.8, 1, new)
    if case.get("pad") and B > 2:
        new[r.randint(1, B)] = 0
    new[0] = new_top
    lens = r.randint(case["max_len"] // 2, case["max_len"] + 1, B)
    lens[0] = case["max_len"]
    if case["op"] == "tables" and B > 4:
        lens[r.randint(1, B)] = 0
    return lens, new


def _gpu(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def _pages(case, seed):
    """A paged cache's geometry: each request's pages in an order without a pattern."""
    lens, new = _lengths(case)
    P = case["page"]
    had, need = -(-lens // P), -(-(lens + new) // P)
    width = int(need.max())
    r = np.random.RandomState((seed + 7) % (1 << 31))
    NB = int(need.sum()) + 3
    ids = r.permutation(NB)
    return lens, new, had, need, width, NB, ids


def _tables_state(case, seed):
    lens, new, had, need, width, NB, ids = _pages(case, seed)
    B = case["B"]
    held = np.arange(width)[None, :] < had[:, None]
    table = np.full((B, width), -1, np.int64)
    table[held] = ids[:int(had.sum())]
    free = np.concatenate([np.full(5, -7), ids[int(had.sum()):]])  # the first five are used already
    return dict(case=case, table=_gpu(table), lens=_gpu(lens), new=_gpu(new), free=_gpu(free), head=_gpu(np.array([5])),
                tokens=int(new.sum()) + case["pad"])


def _encode(x, dims):
    """E4M3 codes and block exponents of float x, blocks spanning `dims`; torch's own conversion."""
    amax = x.abs().amax(dims, keepdim=True)
    m, e = torch.frexp(amax)
    X = (e - 9 + (m > 0.875).to(e.dtype)).clamp(-126, 127)
    codes = torch.ldexp(x, -X).clamp(-448.0, 448.0).to(E4M3)
    byte = torch.where(amax > 0, X + 127, torch.zeros_like(X)).to(torch.uint8)
    return codes, byte


def _cache(case, NB, gen):
    """K or V pages [NB, H, page, D] with the magnitudes differing by page and head, and their scales."""
    shape = (NB, case["H"], case["page"], case["D"])
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.exp2(torch.randn((NB, case["H"], 1, 1), generator=gen, device="cuda"))
    codes, byte = _encode(x, (2, 3))
    return codes.view(torch.uint8), byte.reshape(NB, case["H"])


def _full_table(B, width, need, ids):
    table = np.full((B, width), -1, np.int64)
    table[np.arange(width)[None, :] < need[:, None]] = ids[:int(need.sum())]
    return table


def _store_state(case, seed):
    lens, new, had, need, width, NB, ids = _pages(case, seed)
    P, B = case["page"], case["B"]
    table = _full_table(B, width, need, ids)
    slots = [table[b, (lens[b] + np.arange(new[b])) // P] * P + (lens[b] + np.arange(new[b])) % P for b in range(B)]
    slots = np.concatenate(slots + [np.full(case["pad"], -1)])
    gen = torch.Generator("cuda").manual_seed(seed)
    T, HD = len(slots), case["H"] * case["D"]
    # k and v are two slices of one projection's output
    kv = (torch.randn((T, 2 * HD), generator=gen, device="cuda") *
          torch.exp2(torch.randn((T, 1), generator=gen, device="cuda"))).to(torch.bfloat16)
    kc, ks = _cache(case, NB, gen)
    vc, vs = _cache(case, NB, gen)
    return dict(case=case, k=kv[:, :HD].view(T, case["H"], case["D"]), v=kv[:, HD:].view(T, case["H"], case["D"]),
                slots=_gpu(slots), kc=kc, ks=ks, vc=vc, vs=vs)


def _attn_state(case, seed):
    lens, new, had, need, width, NB, ids = _pages(case, seed)
    H, G, D, B = case["H"], case["G"], case["D"], case["B"]
    gen = torch.Generator("cuda").manual_seed(seed)
    T = int(new.sum()) + case["pad"]
    # q is the first slice of a fused projection's output
    qkv = (torch.randn((T, (H * G + 2 * H) * D), generator=gen, device="cuda") * 1.5).to(torch.bfloat16)
    kc, ks = _cache(case, NB, gen)
    vc, vs = _cache(case, NB, gen)
    return dict(case=case, q=qkv[:, :H * G * D].view(T, H * G, D), kc=kc, ks=ks, vc=vc, vs=vs,
                table=_gpu(_full_table(B, width, need, ids)), lens=_gpu(lens),
                cu=_gpu(np.concatenate([[0], np.cumsum(new)])), max_new=int(new.max()),
                max_len=int((lens + new).max()), out=torch.zeros((T, H * G, D), dtype=torch.bfloat16, device="cuda"))


def _norm_state(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    T, K = case["T"], case["K"]
    big = 1 + 15 * (torch.rand(K, generator=gen, device="cuda") < 0.003).float()  # a few channels stand out
    x = (torch.randn((T, K), generator=gen, device="cuda") * big).to(torch.bfloat16)
    r = (torch.randn((T, K), generator=gen, device="cuda") * 2 * big).to(torch.bfloat16) if case["residual"] else None
    w = (1 + 0.2 * torch.randn(K, generator=gen, device="cuda")).to(torch.bfloat16)
    return dict(case=case, x=x, r=r, w=w)


def _tc_layout(s):
    """[rows, cols] scale bytes -> 128 x 4 atoms, flat, padded with 0."""
    rows, cols = s.shape
    R, C = -(-rows // 128), -(-cols // 4)
    p = torch.zeros((R * 128, C * 4), dtype=torch.uint8, device=s.device)
    p[:rows, :cols] = s
    return p.view(R, 4, 32, C, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _tc_rows(flat, rows, cols):
    """The inverse of _tc_layout."""
    R, C = -(-rows // 128), -(-cols // 4)
    return flat.view(R, C, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R * 128, C * 4)[:rows, :cols]


def _matvec_state(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    M, N, K, nv = case["M"], case["N"], case["K"], case["fmt"] == "nvfp4"
    w = torch.randn((N, K), generator=gen, device="cuda") * 0.02
    blk = 16 if nv else 32
    wb = w.view(N, K // blk, blk)
    amax = wb.abs().amax(2)
    if nv:
        g = (amax.max() / 2688.0).reshape(1)
        sf = (amax / 6.0 / g).clamp(max=448.0).to(E4M3)
        step, sf = sf.float() * g, sf.view(torch.uint8)
    else:
        g = None
        e = torch.frexp(amax)[1] - 3
        step, sf = torch.exp2(e.float()), (e + 127).to(torch.uint8)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    t = wb / step[..., None].clamp_min(1e-30)
    code = torch.bucketize(t.abs(), mids).to(torch.uint8) | ((t < 0).to(torch.uint8) << 3)
    code = code.view(N, K)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    x = torch.randn((M, K), generator=gen, device="cuda")
    x = x * (1 + 15 * (torch.rand(K, generator=gen, device="cuda") < 0.003).float())
    xs = None
    if case["x8"]:
        xc, xb = _encode(x.view(M, K // 32, 32), (2,))
        x, xs = xc.view(torch.uint8).view(M, K), _tc_layout(xb.view(M, K // 32))
    else:
        x = x.to(torch.bfloat16)
    return dict(case=case, x=x, xs=xs, codes=codes.contiguous(), scales=_tc_layout(sf), g=g)


def prepare(case, seed):
    return {"tables": _tables_state, "store": _store_state, "attn": _attn_state, "norm": _norm_state,
            "matvec": _matvec_state}[case["op"]](case, seed)


# ---------------------------------------------------------------- the framework's calls
def _own_tables(s):
    import mxfp4_microscaled_bit_b200 as fl
    cu, slots, head = fl.kv_block_tables(s["table"], s["lens"], s["new"], s["free"], s["head"], s["case"]["page"],
                                         max_tokens=s["tokens"])
    return s["table"], cu, slots, head


def _own_store(s):
    import mxfp4_microscaled_bit_b200 as fl
    fl.kv_fp8_store(s["k"], s["v"], s["slots"], (s["kc"], s["ks"]), (s["vc"], s["vs"]))
    return s["kc"].view(E4M3), s["ks"].view(E8M0), s["vc"].view(E4M3), s["vs"].view(E8M0)


def _own_attn(s):
    import mxfp4_microscaled_bit_b200 as fl
    return fl.kv_fp8_attention(s["q"], (s["kc"], s["ks"]), (s["vc"], s["vs"]), s["table"], s["lens"], s["cu"],
                               max_new=s["max_new"], max_len=s["max_len"], out=s["out"])


def _own_norm(s):
    import mxfp4_microscaled_bit_b200 as fl
    codes, scales, summed = fl.rmsnorm_mxfp8(s["x"], s["w"], s["r"], eps=1e-6, hadamard=s["case"]["hadamard"])
    return codes.view(E4M3), scales.view(E8M0), summed


def _own_matvec(s):
    import mxfp4_microscaled_bit_b200 as fl
    if s["case"]["fmt"] == "nvfp4":
        return fl.nvfp4_matvec(s["x"], s["codes"], s["scales"], s["g"], x_scales=s["xs"],
                               hadamard=s["case"]["hadamard"])
    return fl.mxfp4_matvec(s["x"], s["codes"], s["scales"], x_scales=s["xs"], hadamard=s["case"]["hadamard"])


# ---------------------------------------------------------------- the plain forms
def _plain_tables(s):
    P, table, lens, new, free = s["case"]["page"], s["table"].long(), s["lens"].long(), s["new"].long(), s["free"].long()
    width = table.shape[1]
    had, need = (lens + P - 1) // P, (lens + new + P - 1) // P
    add = need - had
    zero = torch.zeros(1, dtype=torch.long, device=lens.device)
    cu = torch.cat([zero, torch.cumsum(new, 0)])
    first = torch.cumsum(add, 0) - add + s["head"].long()
    col = torch.arange(width, device=lens.device)
    fresh = (col >= had[:, None]) & (col < need[:, None])
    at = (first[:, None] + col - had[:, None]).clamp(0, free.numel() - 1)
    table = torch.where(fresh, free[at], table)
    t = torch.arange(s["tokens"], device=lens.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp_max(lens.numel() - 1)
    p = lens[b] + t - cu[b]
    slots = table[b, (p // P).clamp_max(width - 1)] * P + p % P
    slots = torch.where(t < cu[-1], slots, torch.full_like(slots, -1))
    return table.int(), cu.int(), slots.int(), (s["head"].long() + add.sum()).int()


def _plain_append(new_rows, slots, codes, byte, P):
    """One of K and V.  A page whose first new row is its row 0 starts afresh; any other keeps the
    larger of its old exponent and the new rows', its old rows re-encoded to it."""
    NB, H, _, D = codes.shape
    live = slots >= 0
    page, row = (slots.clamp_min(0) // P).long(), (slots.clamp_min(0) % P).long()
    x = new_rows.float()
    amax = torch.where(live[:, None], x.abs().amax(2), torch.zeros_like(x[:, :, 0]))
    top = torch.zeros((NB, H), device=x.device).scatter_reduce(0, page[:, None].expand(-1, H), amax, "amax")
    low = torch.full((NB,), P, device=x.device, dtype=torch.long).scatter_reduce(
        0, page, torch.where(live, row, torch.full_like(row, P)), "amin")
    m, e = torch.frexp(top)
    X = (e - 9 + (m > 0.875).to(e.dtype)).clamp(-126, 127) + 127
    X = torch.where(top > 0, X, torch.zeros_like(X))
    at = torch.nonzero(low < P)[:, 0]  # the pages with new rows
    old, low, X = byte[at].int(), low[at], X[at]
    both = torch.where(low[:, None] > 0, torch.maximum(old, X), X)
    keep = torch.arange(P, device=x.device)[None, :] < low[:, None]  # rows before the first new one
    held = codes[at]
    again = torch.ldexp(held.view(E4M3).float(), (old - both).clamp_max(0)[:, :, None, None]).to(E4M3).view(torch.uint8)
    codes[at] = torch.where(keep[:, None, :, None], again, held)
    byte[at] = both.to(torch.uint8)
    enc = torch.ldexp(x, 127 - byte[page].int()[:, :, None].clamp_min(1)).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
    t = torch.nonzero(live)[:, 0]
    codes[page[t], :, row[t]] = enc[t]


def _plain_store(s):
    _plain_append(s["k"], s["slots"], s["kc"], s["ks"], s["case"]["page"])
    _plain_append(s["v"], s["slots"], s["vc"], s["vs"], s["case"]["page"])
    return s["kc"].view(E4M3), s["ks"].view(E8M0), s["vc"].view(E4M3), s["vs"].view(E8M0)


def _plain_attn(s):
    c, table = s["case"], s["table"].long()
    H, G, D, P, B = c["H"], c["G"], c["D"], c["page"], c["B"]
    L, Tm = table.shape[1] * P, s["max_new"]
    new = (s["cu"][1:] - s["cu"][:-1]).long()

    def rows(codes, byte):  # [B, H, L, D] in 32 bits
        x = codes.view(E4M3)[table.clamp_min(0)].float()
        x = x * torch.exp2(byte[table.clamp_min(0)].float() - 127.0)[..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, H, L, D)

    i = torch.arange(Tm, device=table.device)
    at = (s["cu"][:-1].long()[:, None] + i).clamp_max(s["q"].shape[0] - 1)
    q = s["q"][at].float().view(B, Tm, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * Tm, D)
    score = torch.matmul(q, rows(s["kc"], s["ks"]).transpose(2, 3)).view(B, H, G, Tm, L) / math.sqrt(D)
    seen = torch.arange(L, device=table.device) <= (s["lens"].long()[:, None] + i)[..., None]  # [B, Tm, L]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    score = torch.exp(score - score.amax(-1, keepdim=True))
    score = score / score.sum(-1, keepdim=True)
    v = rows(s["vc"], s["vs"])
    held = torch.arange(L, device=table.device) < (s["lens"].long() + new)[:, None]
    v = torch.where(held[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(score.view(B, H, G * Tm, L), v).view(B, H, G, Tm, D).permute(0, 3, 1, 2, 4)
    live = i[None] < new[:, None]
    out = torch.zeros_like(s["out"])
    out[at[live]] = o.reshape(B, Tm, H * G, D)[live].to(torch.bfloat16)
    return out


def _sylvester(b, device, dtype):
    h = torch.ones((1, 1), device=device, dtype=dtype)
    while h.shape[0] < b:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(b)


def _rotate(x, b):
    return x if not b else (x.view(-1, b) @ _sylvester(b, x.device, x.dtype)).view(x.shape)


def _plain_norm(s):
    T, K = s["x"].shape
    summed = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(torch.bfloat16)
    v = summed.float()
    n = v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6) * s["w"].float()
    codes, byte = _encode(_rotate(n, s["case"]["hadamard"]).view(T, K // 32, 32), (2,))
    return codes.view(T, K), _tc_layout(byte.view(T, K // 32)).view(E8M0), summed


def _plain_matvec(s):
    c = s["case"]
    N, K, nv = c["N"], c["K"], c["fmt"] == "nvfp4"
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device="cuda")
    w = grid[torch.stack([s["codes"] & 15, s["codes"] >> 4], 2).view(N, K).int()]
    sf = _tc_rows(s["scales"], N, K // (16 if nv else 32))
    sf = sf.contiguous().view(E4M3).float() * s["g"] if nv else torch.exp2(sf.float() - 127.0)
    w = (w.view(N, sf.shape[1], -1) * sf[..., None]).view(N, K)
    if c["x8"]:
        x = s["x"].view(E4M3).float().view(c["M"], K // 32, 32)
        x = (x * torch.exp2(_tc_rows(s["xs"], c["M"], K // 32).float() - 127.0)[..., None]).view(c["M"], K)
    else:
        x = _rotate(s["x"].float(), c["hadamard"])
    return (x @ w.t()).to(torch.bfloat16)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tables": _own_tables, "store": _own_store, "attn": _own_attn, "norm": _own_norm,
                "matvec": _own_matvec}[op](state)
    return {"tables": _plain_tables, "store": _plain_store, "attn": _plain_attn, "norm": _plain_norm,
            "matvec": _plain_matvec}[op](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("tables", "store", "attn"):
        lens, new, had, need, width, NB, ids = _pages(case, 0)
    if op == "tables":
        T, fresh, B = int(new.sum()), int((need - had).sum()), case["B"]
        # lengths in; block ids from the free list into the table; the table's last blocks in, slots and offsets out
        return dict(bytes=4 * (2 * B + 2 * fresh + B + T + case["pad"] + B + 1 + 2), flops=T)
    if op == "store":
        n = int(new.sum()) * case["H"] * case["D"]
        return dict(bytes=2 * 3 * n + 4 * int(new.sum()) + 4 * int((need - lens // case["page"]).sum()) * case["H"],
                    flops=2 * 2 * n)
    if op == "attn":
        H, G, D = case["H"], case["G"], case["D"]
        seen = int((lens * new + new * (new + 1) // 2).sum())
        keys = int((lens + new).sum())
        return dict(bytes=2 * keys * H * D + 2 * int(need.sum()) * H + 4 * int(need.sum()) + 2 * 2 * int(new.sum()) * H * G * D,
                    flops=4 * seen * H * G * D)
    if op == "norm":
        n = case["T"] * case["K"]
        return dict(bytes=n * (2 + 1) + n / 32 + 2 * case["K"] + (4 * n if case["residual"] else 0), flops=6 * n)
    M, N, K = case["M"], case["N"], case["K"]
    w = N * K / 2 + N * K / (16 if case["fmt"] == "nvfp4" else 32)
    return dict(bytes=w + M * K * (1 + 1 / 32 if case["x8"] else 2) + 2 * M * N, flops=2 * M * N * K)


# ---------------------------------------------------------------- the definitions in 64 bits
def _e4m3_64(u):
    """Values of E4M3 bytes: exponent bias 7, three mantissa bits, subnormals in steps of 2^-9."""
    u = u.to(torch.int64)
    e, m = (u >> 3) & 15, (u & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.pow(torch.tensor(2.0, device=u.device, dtype=torch.float64), (e - 7).double()), m / 512)
    v = torch.where((u & 127) == 127, torch.full_like(v, math.nan), v)
    return torch.where(u > 127, -v, v)


def _least_exponent(amax):
    """The least integer X >= -126 with amax <= 448 * 2^X, from the logarithm and then put right."""
    X = torch.floor(torch.log2(amax.clamp_min(1e-300) / 448.0)).clamp(-126, 127)
    X = torch.where(448.0 * torch.exp2(X) < amax, X + 1, X)
    return torch.where(448.0 * torch.exp2(X) < amax, X + 1, X)


def _exact_store(s):
    P, out = s["case"]["page"], []
    slots = s["slots"].tolist()
    runs, t = [], 0
    while t < len(slots):  # runs of new rows within a page
        n = 1
        while slots[t] >= 0 and t + n < len(slots) and slots[t + n] == slots[t] + n and (slots[t] + n) % P:
            n += 1
        if slots[t] >= 0:
            runs.append((t, n, slots[t] // P, slots[t] % P))
        t += n
    if len(runs) > 3000:
        return None
    for x, codes, byte in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        c, b = _e4m3_64(codes), byte.double()
        for t, n, page, row in runs:
            new = x[t:t + n].double()  # [n, H, D]
            top = new.abs().amax((0, 2))
            X = torch.where(top > 0, _least_exponent(top) + 127, torch.zeros_like(top))
            if row:
                both = torch.maximum(X, byte[page].double())
                c[page, :, :row] *= torch.exp2(byte[page].double() - both)[:, None, None]
                X = both
            b[page] = X
            c[page, :, row:row + n] = (new * torch.exp2(127 - X.clamp_min(1))[None, :, None]).transpose(0, 1)
        out += [c, torch.exp2(b - 127)]
    return tuple(out)


def _exact_attn(s):
    c = s["case"]
    H, G, D, P = c["H"], c["G"], c["D"], c["page"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    for b in range(c["B"]):
        n = cu[b + 1] - cu[b]
        if not n:
            continue
        L = lens[b] + n
        pages = s["table"][b, :-(-L // P)].long()
        for h in range(H):
            k, v = ((_e4m3_64(codes[pages, h]) * torch.exp2(byte[pages, h].double() - 127)[:, None, None]).view(-1, D)[:L]
                    for codes, byte in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            q = s["q"][cu[b]:cu[b + 1], h * G:(h + 1) * G].double()  # [n, G, D]
            w = torch.einsum("igd,ld->igl", q, k) * D ** -0.5
            later = torch.arange(L, device="cuda")[None, :] > lens[b] + torch.arange(n, device="cuda")[:, None]
            w = torch.softmax(w.masked_fill(later[:, None], -math.inf), -1)
            out[cu[b]:cu[b + 1], h * G:(h + 1) * G] = torch.einsum("igl,ld->igd", w, v)
    return out


def _hadamard_64(x, b):
    """Butterflies over blocks of b, in 64 bits."""
    if not b:
        return x
    y, h = x.reshape(-1, b).clone(), 1
    while h < b:
        y = y.view(-1, b // (2 * h), 2, h)
        y = torch.stack([y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]], 2).reshape(-1, b)
        h *= 2
    return (y / b ** 0.5).reshape(x.shape)


def _exact_norm(s):
    T, K = s["x"].shape
    v = s["x"].double() + (0 if s["r"] is None else s["r"].double())
    summed, v = v, v.to(torch.bfloat16).double()  # the sum's own rounding is part of the definition
    n = v / torch.sqrt((v * v).sum(1, keepdim=True) / K + 1e-6) * s["w"].double()
    n = _hadamard_64(n, s["case"]["hadamard"]).view(T, K // 32, 32)
    top = n.abs().amax(2)
    X = _least_exponent(top)
    byte = torch.where(top > 0, X + 127, torch.zeros_like(X)).to(torch.uint8)
    return (n * torch.exp2(-X)[..., None]).view(T, K), torch.exp2(_tc_layout(byte).double() - 127), summed


def _exact_matvec(s):
    c = s["case"]
    M, N, K = c["M"], c["N"], c["K"]
    blk = 16 if c["fmt"] == "nvfp4" else 32

    def scale_at(flat, rows, cols):  # the byte of scale (r, c) by the layout's formula
        r, k = torch.arange(rows, device="cuda")[:, None], torch.arange(cols, device="cuda")[None, :]
        return flat[((r // 128) * (-(-cols // 4)) + k // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4]

    w = torch.empty((N, K), dtype=torch.float64, device="cuda")
    for half in (0, 1):
        u = ((s["codes"] >> (4 * half)) & 15).to(torch.int64)
        e, m = (u >> 1) & 3, (u & 1).double()
        mag = torch.where(e > 0, (1 + m / 2) * torch.exp2((e - 1).double()), m / 2)
        w[:, half::2] = torch.where(u > 7, -mag, mag)
    sf = scale_at(s["scales"], N, K // blk)
    sf = _e4m3_64(sf) * s["g"].double() if blk == 16 else torch.exp2(sf.double() - 127)
    w.view(N, K // blk, blk).mul_(sf[..., None])
    if c["x8"]:
        x = _e4m3_64(s["x"]) * torch.exp2(scale_at(s["xs"], M, K // 32).double() - 127).repeat_interleave(32, 1)
    else:
        x = _hadamard_64(s["x"].double(), c["hadamard"])
    return x @ w.t()


def exact(case, seed):
    if case["op"] == "tables":  # whole numbers only
        return None
    s = prepare(case, seed)
    return {"store": _exact_store, "attn": _exact_attn, "norm": _exact_norm, "matvec": _exact_matvec}[case["op"]](s)
