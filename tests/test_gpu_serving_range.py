"""The serving operators where values lie far apart: dominant keys, pages of zeros, block scales and
channels many binades from each other.  Plain 64-bit forms as in test_gpu_serving."""
import numpy as np
import pytest
import torch

import mxfp4_microscaled_bit_b200 as fl
import serving_ref as ref
from gpu_util import DEV, status_ok
from test_gpu_serving import BF16, F16, F32, attention_case, gpu, u8, within

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention
def weight_floor(q, kc, kb, vc, vb, table, lens, cu, P, scale):
    """The absolute part of the weights' f16 rounding.  A weight and its page's value scale make one
    number W = p 2^Xv, held relative to the row's largest, which sits in f16 at 2^14 where a request has
    up to 16 (token, head) rows and at 2^6 or above where it has more: half a step of a subnormal f16
    is 2^-25, so every W is within 2^-39 (2^-31) of the largest, and meets |code|.  A page of zero
    values (byte 0) has a part in the largest 2^-24 below the pages with values at most."""
    T, HQ, D = q.shape
    NP, H = kb.shape
    G = HQ // H
    floor = np.zeros((T, HQ, D))
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        L = lens[b] + n
        if n <= 0:
            continue
        part = 2.0 ** (-39 if n * G <= 16 else -31)
        pages = table[b, :-(-L // P)]
        for h in range(H):
            k = ref.cache_values(kc[pages, h], kb[pages, h]).reshape(-1, D)[:L]
            code = np.abs(ref.E4M3[vc[pages, h]]).reshape(-1, D)[:L]
            x = np.repeat(vb[pages, h].astype(np.float64) - 127, P)[:L]
            held = x > -127
            for i in range(n):
                see = np.arange(L) <= lens[b] + i
                if not (see & held).any():
                    continue
                xs = np.where(held, x, x[see & held].max() - 24)
                for j in range(h * G, (h + 1) * G):
                    s = scale * (k[see] @ q[cu[b] + i, j])
                    p = np.exp(s - s.max())
                    W = p / p.sum() * 2.0 ** xs[see]
                    floor[cu[b] + i, j] = part * W.max() * code[see].sum(0)
    return floor


def range_check(q, caches, table, lens, cu, P):
    (kc, kb), (vc, vb) = caches
    T, HQ, D = q.shape
    n = np.diff(cu)
    out = torch.full((T, HQ, D), 123.0, dtype=torch.bfloat16, device=DEV)
    fl.kv_fp8_attention(q.to(DEV), (u8(kc), u8(kb)), (u8(vc), u8(vb)), gpu(table), gpu(lens), gpu(cu),
                        max_new=int(n.max()), max_len=int((lens + n).max()), out=out)
    status_ok()
    a = ref.f64(q), kc, kb, vc, vb, table, lens, cu, P, D ** -0.5
    want, spread, dots = ref.attention(*a)
    mine = ~np.isnan(want)
    got = ref.f64(out)
    assert (got[~mine] == 123.0).all(), "rows of no request were written"
    L = int((lens + n).max())
    # a weight's relative error as in test_gpu_serving's attention_check, and the floor
    tol = (2 * ((D + 6) * F32 * dots + 2.0 ** -21) + F16 + 2 * L * F32) * spread + weight_floor(*a)
    within(got[mine], want[mine], (tol * (1 + BF16) + BF16 * np.abs(want))[mine], "attention")


def sink(q, caches, table, P, G, D, row, gap, whole_page):
    """Key `row` of request 0 with a logit about `gap` above every other's and a zero value; with
    whole_page its page holds no other values either (byte 0)."""
    (kc, kb), (vc, vb) = caches
    H = kb.shape[1]
    page, at = table[0, row // P], row % P
    kc[:, :, :, 0] = 0
    kc[page, :, at] = 0
    kc[page, :, at, 0] = 0x7E
    for h in range(H):
        top = 448.0 * 2.0 ** (float(kb[page, h]) - 127)
        q[:, h * G:(h + 1) * G, 0] = gap / (top * D ** -0.5)
    vc[:] &= 0x7F  # values of one sign: what is lost does not average out
    vc[page, :, at] = 0
    if whole_page:
        vc[page], vb[page] = 0, 0


@pytest.mark.parametrize("whole_page", [False, True])
@pytest.mark.parametrize("D,G,P,L,new,gap", [
    (128, 4, 16, 4000, 1, 20.0),    # the split kernel, its splits joined in a cluster
    (64, 4, 64, 20000, 1, 20.0),    # and through the workspace
    (128, 8, 32, 1500, 2, 20.0),    # 16 rows
    (64, 2, 16, 300, 40, 18.0),     # the many-row kernel, a tile's keys in one CTA
    (128, 4, 64, 4000, 70, 18.0)])  # and shared among CTAs
def test_attention_of_a_dominant_key_without_a_value(D, G, P, L, new, gap, whole_page):
    q, caches, table, lens, cu = attention_case(1, 2, G, D, P, [L], [new], seed=L, sigma=0.4, spread=0.3)
    sink(q, caches, table, P, G, D, 5, gap, whole_page)
    range_check(q, caches, table, lens, cu, P)


@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("big", [2.0 ** 10, 2.0 ** 18, 2.0 ** 24])
def test_attention_of_scores_whose_rounding_passes_the_weights_room(new, big):
    """Scores so large that binary32 rounds them by whole binades: no weight becomes infinite, and
    the answer stays among the values."""
    q, ((kc, kb), (vc, vb)), table, lens, cu = attention_case(1, 2, 4, 64, 32, [500], [new], seed=6)
    out = fl.kv_fp8_attention((q.float() * big).to(torch.bfloat16).to(DEV), (u8(kc), u8(kb)), (u8(vc), u8(vb)),
                              gpu(table), gpu(lens), gpu(cu), max_new=new, max_len=500 + new)[:new]
    status_ok()
    held = np.nan_to_num(np.abs(ref.cache_values(vc, vb))).max()
    assert bool(out.isfinite().all()) and float(out.abs().max()) <= held * (1 + 2 * BF16)


@pytest.mark.parametrize("v_shift", [-30, -60, 40])
@pytest.mark.parametrize("L,new,zero", [
    (170, 1, [1, 4]), (170, 70, [1, 4]), (90, 5, [0]), (90, 90, [0]),
    (3000, 1, list(range(40))), (3000, 60, list(range(40))),  # whole splits, and shared parts, of zero pages
    (3000, 1, list(range(100, 188))), (700, 33, [44, 45]),    # the last ones, which some rows see in part
    (25000, 1, list(range(3, 1500)))])
def test_attention_zero_pages_beside_values_of_any_magnitude(L, new, zero, v_shift):
    q, ((kc, kb), (vc, vb)), table, lens, cu = attention_case(1, 1, 4, 64, 16, [L], [new], seed=L + new)
    vb = (vb.astype(int) + v_shift).astype(np.uint8)
    vc[table[0, zero]], vb[table[0, zero]] = 0, 0
    range_check(q, ((kc, kb), (vc, vb)), table, lens, cu, 16)


@pytest.mark.parametrize("new", [1, 50])
def test_attention_zero_pages_between_pages_far_apart(new):
    """The zero pages come before the pages of the smallest values, and after."""
    q, ((kc, kb), (vc, vb)), table, lens, cu = attention_case(2, 2, 4, 128, 16, [600, 300], [new, new], seed=2, sigma=0.5)
    vb = vb.astype(int)
    for b in range(2):
        vb[table[b, 8:]] -= 22
        for p in (1, 12):
            vc[table[b, p]], vb[table[b, p]] = 0, 0
    range_check(q, ((kc, kb), (vc, vb.astype(np.uint8))), table, lens, cu, 16)


@pytest.mark.parametrize("new", [1, 3, 40])
@pytest.mark.parametrize("far", [2.0 ** 12, 2.0 ** 20, 2.0 ** -20])
def test_attention_of_a_query_whose_channels_are_far_apart(new, far):
    """One channel of q away from the others, where the keys have nothing (or everything) in it."""
    q, ((kc, kb), (vc, vb)), table, lens, cu = attention_case(1, 2, 4, 64, 32, [200], [new], seed=8)
    q[:, :, 0] = far
    if far > 1:
        kc[:, :, :, 0] = 0
    range_check(q, ((kc, kb), (vc, vb)), table, lens, cu, 32)


# ------------------------------------------------------------------ blocks of nothing finite
@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan")])
def test_append_and_attention_of_pages_without_a_finite_value(what):
    """Infinities saturate at 448 times the least scale there is, and shrink to nothing when the
    page's scale grows; a page of them, or of NaN, is not taken for one of zeros."""
    H, P, D = 2, 16, 64
    caches = [(torch.full((2, H, P, D), 0x55, dtype=torch.uint8, device=DEV),
               torch.full((2, H), 9, dtype=torch.uint8, device=DEV)) for _ in range(2)]
    x = torch.zeros(1, H, D, dtype=torch.bfloat16, device=DEV)
    x[:, :, ::3] = what
    k = torch.zeros_like(x)
    fl.kv_fp8_store(k, x, gpu([16]), *caches)
    status_ok()
    codes, byte = caches[1][0][1, :, 0].cpu(), caches[1][1][1].cpu()
    bad = 0x7F if what != what else 0x7E if what > 0 else 0xFE
    assert (byte == 1).all() and not codes[:, 1::3].any()
    assert ((codes[:, ::3] & 0x7F) == 0x7F).all() if what != what else (codes[:, ::3] == bad).all()
    assert not caches[0][1][1].any() and not caches[0][0][1, :, 0].any()  # zeros: byte 0
    for new in (1, 40):  # one row of keys, seen by one token or by the first of many
        q = torch.ones(new, 2 * H, D, dtype=torch.bfloat16, device=DEV)
        out = fl.kv_fp8_attention(q, *caches, gpu([[1, 0, 0, 0]]), gpu([0]), gpu([0, new]), max_new=new, max_len=64)[0]
        status_ok()
        want = 448.0 * 2.0 ** -126 * (1 if what > 0 else -1)
        got = ref.f64(out)
        assert np.isnan(got[:, ::3]).all() if what != what else (np.abs(got[:, ::3] - want) <= BF16 * abs(want)).all()
        assert not got[:, 1::3].any()
    y = torch.randn(1, H, D, device=DEV).to(torch.bfloat16)
    fl.kv_fp8_store(k, y, gpu([17]), *caches)
    status_ok()
    codes, byte = caches[1][0][1, :, 0].cpu(), caches[1][1][1].cpu()
    assert byte.tolist() == ref.block_byte(np.abs(ref.f64(y))[0].max(1)).tolist()
    assert ((codes[:, ::3] & 0x7F) == 0x7F).all() if what != what else not (codes & 0x7F).any()


def test_norm_of_a_block_without_a_finite_value():
    x = torch.randn(3, 128, device=DEV).abs().to(torch.bfloat16) + 1
    x[2, 96:] = 0
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    w[32:64] = float("inf")
    w[64:96] = float("nan")
    c, s, _ = fl.rmsnorm_mxfp8(x, w)
    status_ok()
    byte = ref.tc_rows(s.cpu().numpy(), 3, 4)
    assert (byte[:, 1:3] == 1).all() and (c[:, 32:64] == 0x7E).all() and (c[:, 64:96] & 127 == 127).all()
    assert byte[2, 3] == 0 and not c[2, 96:].any() and (byte[:, 0] > 1).all()


# ------------------------------------------------------------------ matvec
def scale_layout(byte):
    """[rows, cols] scale bytes in the tensor-core layout."""
    rows, cols = byte.shape
    katoms = -(-cols // 4)
    flat = np.zeros(fl.scale_bytes(rows, cols), np.uint8)
    r, c = np.arange(rows)[:, None], np.arange(cols)[None]
    flat[((r // 128) * katoms + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4] = byte
    return flat


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,low,high", [(1, 16, 21), (5, 16, 30), (16, 25, 36), (3, 0, 60)])
def test_matvec_of_8_bit_rows_whose_block_scales_lie_far_apart(fmt, M, low, high):
    """The largest block of 256 values meets zero weights: the answer is the others'."""
    N, K = 40, 768
    rng = np.random.default_rng(M + high)
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    x = rng.integers(0, 256, (M, K), dtype=np.uint8)
    x[(x & 127) == 127] = 1
    byte = 150 - rng.integers(low, high + 1, (M, K // 32))
    for chunk in range(3):
        block = 8 * chunk + [0, 5, 7][chunk]
        byte[:, block] = 150
        codes[:, block * 16:block * 16 + 16] = 0
    if fmt == "nvfp4":
        sb, g = rng.integers(40, 100, (N, K // 16)), torch.tensor([0.25], device=DEV)
        y = fl.nvfp4_matvec(u8(x), u8(codes), u8(scale_layout(sb)), g, x_scales=u8(scale_layout(byte)))
    else:
        sb = rng.integers(115, 122, (N, K // 32))
        y = fl.mxfp4_matvec(u8(x), u8(codes), u8(scale_layout(sb)), x_scales=u8(scale_layout(byte)))
    status_ok()
    W = np.abs(ref.weight(codes, scale_layout(sb), fmt, 0.25))
    xv = ref.E4M3[x] * np.repeat(2.0 ** (byte - 127.0), 32, 1)
    want, mag = xv @ ref.weight(codes, scale_layout(sb), fmt, 0.25).T, np.abs(xv) @ W.T
    # exact to 2^-21 of the largest scale; else rounded to f16 subnormals, half a step of which is
    # 2^-31 of that scale
    err = np.where(150 - byte <= 21, 0.0, 2.0 ** (150 - 127 - 31)).repeat(32, 1) @ W.T
    tol = (K + 8) * F32 * mag + err
    within(ref.f64(y), want, tol * (1 + BF16) + BF16 * np.abs(want), "8-bit rows")


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("M,low,high", [(1, 20, 36), (4, 24, 36), (11, 0, 36), (16, 30, 36), (2, 36, 45)])
def test_matvec_of_mxfp4_weights_whose_block_scales_lie_far_apart(M, low, high, x8):
    """x is zero in the largest block of 256 values: the answer is the others'."""
    N, K = 150, 512
    rng = np.random.default_rng(M + high)
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    byte = 140 - rng.integers(low, high + 1, (N, K // 32))
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16)
    for block in (3, 15):
        byte[:, block] = 140
        x[:, block * 32:block * 32 + 32] = 0
    if x8:
        xc = ref.e4m3_bytes(ref.f64(x))
        xb = np.full((M, K // 32), 127)
        xv = ref.E4M3[xc]
        y = fl.mxfp4_matvec(u8(xc), u8(codes), u8(scale_layout(byte)), x_scales=u8(scale_layout(xb)))
    else:
        xv = ref.f64(x)
        y = fl.mxfp4_matvec(x.to(DEV), u8(codes), u8(scale_layout(byte)))
    status_ok()
    W = ref.weight(codes, scale_layout(byte), "mxfp4")
    want, mag = xv @ W.T, np.abs(xv) @ np.abs(W).T
    # exact to 2^-36 of the row's largest scale in 256 values, at 2^-37 within half a step of a subnormal
    # f16 under 2^13, 2^-38 of that scale, and nothing is kept of 6 times the scale below
    k = 140 - byte
    far = np.where(k <= 36, 0.0, np.where(k == 37, 2.0 ** -38, 6.0 * 2.0 ** -k))
    tol = (K + 8) * F32 * mag + np.abs(xv) @ (2.0 ** 13 * far).repeat(32, 1).T
    within(ref.f64(y), want, tol * (1 + BF16) + BF16 * np.abs(want), "far MXFP4 scales")


# ------------------------------------------------------------------ tensors that lie between one another
def test_norm_of_column_slices_of_one_buffer():
    """x, the residual and the sum side by side in the rows of one projection's output."""
    rows, cols = 70, 256
    base = torch.randn(rows, 3 * cols + 8, device=DEV).to(torch.bfloat16)
    x, r, s = base[:, :cols], base[:, cols:2 * cols], base[:, 2 * cols + 8:]
    w = torch.randn(cols, device=DEV).to(torch.bfloat16)
    want = fl.rmsnorm_mxfp8(x.contiguous(), w, r.contiguous(), hadamard=32)
    keep = base.clone()
    got = fl.rmsnorm_mxfp8(x, w, r, hadamard=32, summed=s)
    status_ok()
    assert got[2] is s and all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(base[:, :2 * cols + 8], keep[:, :2 * cols + 8])
    with pytest.raises(ValueError, match="overlaps residual"):
        fl.rmsnorm_mxfp8(x, w, r, summed=base[:, 2 * cols - 8:3 * cols - 8])


# ------------------------------------------------------------------ offsets that pass 32 bits
def test_paged_cache_of_more_than_4_gb():
    """The same step on the last pages of a large cache and on a small one: the same bits."""
    H, G, P, D, lens, new = 8, 2, 128, 128, [300, 40], [1, 30]
    far = (1 << 32) // (H * P * D) + 1
    g = torch.Generator(device=DEV).manual_seed(0)
    kv = torch.randn(2, 371, H, D, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn(31, H * G, D, generator=g, device=DEV).to(torch.bfloat16)
    outs = []
    for first in (0, far):
        caches = [(torch.empty((first + 4, H, P, D), dtype=torch.uint8, device=DEV),
                   torch.empty((first + 4, H), dtype=torch.uint8, device=DEV)) for _ in range(2)]
        for codes, scales in caches:
            codes[first:], scales[first:] = 0, 0
        table = gpu(np.array([[2, 0, 3], [1, -1, -1]]) + first * (np.arange(3) < [[3], [1]]))
        p = [np.arange(n) for n in (301, 70)]
        rows = table.cpu().numpy()
        slots = np.concatenate([rows[b, p[b] // P] * P + p[b] % P for b in range(2)])
        fl.kv_fp8_store(kv[0], kv[1], gpu(slots), *caches)
        out = fl.kv_fp8_attention(q, *caches, table, gpu(lens), gpu([0, 1, 31]), max_new=30, max_len=301)
        status_ok()
        outs.append([out] + [t[first:].clone() for c in caches for t in c])
        del caches
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    torch.cuda.empty_cache()


def test_norm_and_matvec_of_more_than_4_gb():
    rows, cols = 70000, 32768
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[-130:] = torch.randn(130, cols, device=DEV).to(torch.bfloat16)
    w = torch.randn(cols, device=DEV).to(torch.bfloat16)
    c, s, _ = fl.rmsnorm_mxfp8(x, w, hadamard=16)
    status_ok()
    cut = rows // 128 * 128 - 128  # whole tiles of the scale layout
    c0, s0, _ = fl.rmsnorm_mxfp8(x[cut:], w, hadamard=16)
    assert torch.equal(c[cut:], c0) and torch.equal(s[cut * cols // 32:], s0)
    del x, c, s
    N, K = (1 << 20) + 3, 8256
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.zeros(fl.scale_bytes(N, K // 32), dtype=torch.uint8, device=DEV)
    codes[-131:] = torch.randint(0, 256, (131, K // 2), device=DEV).to(torch.uint8)
    tail = fl.scale_bytes(131, K // 32)  # the last 131 rows are two tiles
    scales[-tail:] = torch.randint(110, 130, (tail,), device=DEV).to(torch.uint8)
    x = torch.randn(3, K, device=DEV).to(torch.bfloat16)
    y = fl.mxfp4_matvec(x, codes, scales)
    status_ok()
    assert not y[:, :-131].any()
    W = ref.weight(codes[-131:].cpu().numpy(), scales[-tail:].cpu().numpy(), "mxfp4")
    want, mag = ref.f64(x) @ W.T, np.abs(ref.f64(x)) @ np.abs(W).T
    within(ref.f64(y[:, -131:]), want, (K + 8) * F32 * mag * (1 + BF16) + BF16 * np.abs(want), "the last rows")
    torch.cuda.empty_cache()
