"""The serving operators on the GPU against their plain 64-bit forms (serving_ref)."""
import numpy as np
import pytest
import torch

import mxfp4_microscaled_bit_b200 as fl
import serving_ref as ref
from gpu_util import DEV, status_ok

pytestmark = pytest.mark.gpu
OUT_OF_RANGE = 8
BF16, F16, F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24  # half a step, relative


def gpu(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device=DEV)


def u8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def within(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[:3].tolist()}: "
                           f"got {got[bad][:3]} want {want[bad][:3]} tol {np.broadcast_to(tol, bad.shape)[bad][:3]}")


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("rows,cols,had,residual", [
    (1, 32, 0, True), (1, 4096, 16, True), (3, 64, 32, False), (5, 96, 0, True), (129, 1024, 16, True),
    (7, 1056, 32, True), (130, 2880, 0, False), (2, 14336, 32, True), (2, 16416, 16, True), (1, 32768, 0, True)])
def test_norm(rows, cols, had, residual):
    g = torch.Generator().manual_seed(rows * cols + had)
    x = (torch.randn(rows, cols, generator=g) * 3).to(torch.bfloat16)
    r = (torch.randn(rows, cols, generator=g)).to(torch.bfloat16) if residual else None
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(torch.bfloat16)
    x[-1, : min(32, cols - 32) or 1] = 0  # a block of zeros where there is another
    if residual:
        r[-1, : min(32, cols - 32) or 1] = 0
    codes = torch.full((rows, cols), 0xAA, dtype=torch.uint8, device=DEV)
    scales = torch.full((fl.scale_bytes(rows, cols // 32),), 0xEE, dtype=torch.uint8, device=DEV)
    c, s, summed = fl.rmsnorm_mxfp8(x.to(DEV), w.to(DEV), None if r is None else r.to(DEV), eps=1e-5, hadamard=had,
                                    codes=codes, scales=scales)
    status_ok()
    want = x if r is None else (x.float() + r.float()).to(torch.bfloat16)
    assert torch.equal(summed.cpu(), want)
    v = ref.f64(want)
    n = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-5) * ref.f64(w)
    n = ref.hadamard(n, had)
    # the norm's own error: the sum of squares (half counts in its root), the root, two products
    # (3 + 32 in-lane + 10 tree steps at most), and 5 butterfly steps with the scaling
    rel = (45 / 2 + 4) * F32
    mag = np.sqrt((n.reshape(rows, -1, 32) ** 2).sum(2)).repeat(32, 1)  # bounds the butterflies' terms
    err = rel * np.abs(n) + (rel + 7 * F32) * mag * (1 if had else 0)
    byte = ref.tc_rows(s.cpu().numpy(), rows, cols // 32)
    top = np.abs(n).reshape(rows, -1, 32).max(2)
    slack = err.reshape(rows, -1, 32).max(2)
    lo, hi = ref.block_byte(np.maximum(top - slack, 0)), ref.block_byte(top + slack)
    assert ((byte >= lo) & (byte <= hi)).all()
    step = 2.0 ** (np.maximum(byte, 1).astype(np.float64) - 127).repeat(32, 1)
    got = ref.E4M3[c.cpu().numpy()] * step * np.where(byte == 0, 0, 1).repeat(32, 1)
    within(got, n, err * (1 + 2.0 ** -4) + 2.0 ** -4 * np.abs(n) + 2.0 ** -10 * step, "values")
    pad = s.cpu().numpy().copy()  # every byte that is no scale is zero
    katoms = -(-(cols // 32) // 4)
    rr, cc = np.arange(rows)[:, None], np.arange(cols // 32)[None]
    pad[((rr // 128) * katoms + cc // 4) * 512 + (rr % 32) * 16 + (rr % 128) // 32 * 4 + cc % 4] = 0
    assert not pad.any()


def test_norm_in_place_strided_and_repeated():
    rows, cols = 6, 1536
    base = torch.randn(rows, 2 * cols + 8, device=DEV).to(torch.bfloat16)
    x, r = base[:, :cols], torch.randn(rows, cols, device=DEV).to(torch.bfloat16)
    w = torch.randn(cols, device=DEV).to(torch.bfloat16)
    c0, s0, sum0 = fl.rmsnorm_mxfp8(x, w, r, hadamard=16)
    r2 = r.clone()
    c1, s1, sum1 = fl.rmsnorm_mxfp8(x.contiguous(), w, r2, hadamard=16, summed=r2)
    assert sum1 is r2 and torch.equal(sum1, sum0) and torch.equal(c0, c1) and torch.equal(s0, s1)
    x2 = x.clone()
    assert fl.rmsnorm_mxfp8(x2, w, r, hadamard=16, summed=x2)[2] is x2 and torch.equal(x2, sum0)
    with pytest.raises(ValueError, match="overlaps"):
        fl.rmsnorm_mxfp8(x, w, base[:, 8:8 + cols], summed=base[:, 16:16 + cols])
    with pytest.raises(ValueError, match="contiguous rows"):
        fl.rmsnorm_mxfp8(base.t(), w)
    with pytest.raises(ValueError, match="holds"):
        fl.rmsnorm_mxfp8(x, w[:64])
    with pytest.raises(ValueError, match="holds"):
        fl.rmsnorm_mxfp8(x, w, scales=torch.empty(64, dtype=torch.uint8, device=DEV))
    status_ok()


def test_norm_zero_row_and_nan_row():
    x = torch.randn(3, 128, device=DEV).to(torch.bfloat16)
    x[0] = 0
    x[1, 5] = float("nan")
    c, s, _ = fl.rmsnorm_mxfp8(x, torch.ones(128, dtype=torch.bfloat16, device=DEV))
    byte = ref.tc_rows(s.cpu().numpy(), 3, 4)
    assert not c[0].any() and not byte[0].any()  # zeros: zero codes under byte 0
    assert (c[1] & 127 == 127).all()
    alone = fl.rmsnorm_mxfp8(x[2:], torch.ones(128, dtype=torch.bfloat16, device=DEV))[0]
    assert torch.equal(c[2], alone[0])


# ------------------------------------------------------------------ matvec
def weight(N, K, fmt, had, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + N + K)
    return fl.prepare_weight((torch.randn(N, K, generator=g, device=DEV) * 0.05).to(torch.bfloat16), fmt, had)


def matvec_check(y, x, w, codes_err):
    W = ref.weight(w.codes.cpu().numpy(), w.scales.cpu().numpy(), w.fmt, 1.0 if w.g is None else float(w.g.item()))
    want, mag = x @ W.T, np.abs(x) @ np.abs(W).T
    K = x.shape[1]
    # binary32 sums of K products (exact but for the scalings), three scalings, the bf16 rounding
    tol = (K + 8) * F32 * mag + codes_err * mag
    within(ref.f64(y), want, tol * (1 + BF16) + BF16 * np.abs(want), f"matvec {w.fmt} {x.shape}x{W.shape[0]}")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K,rot", [(1, 1, 64, False), (1, 4096, 4096, True), (2, 130, 192, True), (3, 7, 320, False),
                                       (8, 129, 2048, False), (9, 200, 2112, True), (15, 64, 832, False),
                                       (16, 385, 4160, True), (1, 33, 14336, False), (4, 128, 33024, False)])
def test_matvec_bf16(fmt, M, N, K, rot):
    had = (16 if fmt == "nvfp4" else 32) if rot else 0
    w = weight(N, K, fmt, had)
    x = torch.randn(M, K, device=DEV).to(torch.bfloat16)
    y = fl.weight_only_linear(x, w)
    status_ok()
    # rotated activations: one f16 rounding, and 5 butterfly steps and a scaling on terms that
    # add up to at most sqrt(32) of the block's values
    matvec_check(y, ref.hadamard(ref.f64(x), had), w, 0.0)if not rot else matvec_rotated_check(y, x, w, had)
    assert torch.equal(y, fl.weight_only_linear(x, w))  # the same bits


def matvec_rotated_check(y, x, w, had):
    W = ref.weight(w.codes.cpu().numpy(), w.scales.cpu().numpy(), w.fmt, 1.0 if w.g is None else float(w.g.item()))
    xr = ref.hadamard(ref.f64(x), had)
    block = ref.hadamard(np.abs(ref.f64(x)), 0).reshape(x.shape[0], -1, had).sum(2) / np.sqrt(had)
    err = F16 * np.abs(xr) + 7 * F32 * np.repeat(block, had, 1)
    want, mag = xr @ W.T, np.abs(xr) @ np.abs(W).T
    tol = (x.shape[1] + 8) * F32 * mag + err @ np.abs(W).T
    within(ref.f64(y), want, tol * (1 + BF16) + BF16 * np.abs(want), f"rotated matvec {w.fmt}")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (5, 77, 192), (16, 257, 2304)])
def test_matvec_of_the_norms_output(fmt, M, N, K):
    had = 16 if fmt == "nvfp4" else 32
    w = weight(N, K, fmt, had)
    x = torch.randn(M, K, device=DEV).to(torch.bfloat16)
    c, s, _ = fl.rmsnorm_mxfp8(x, torch.ones(K, dtype=torch.bfloat16, device=DEV), hadamard=had)
    y = fl.weight_only_linear(c, w, x_scales=s)
    status_ok()
    byte = ref.tc_rows(s.cpu().numpy(), M, K // 32)
    xv = ref.E4M3[c.cpu().numpy()] * np.repeat(2.0 ** (byte.astype(np.float64) - 127), 32, 1)
    matvec_check(y, xv, w, 0.0)


def test_matvec_far_scales_and_non_finite_rows():
    # MXFP4 scales over most of the exponent range, activations from 1e-30 to 1e30
    N, K = 40, 512
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    flat = np.zeros(fl.scale_bytes(N, K // 32), np.uint8)
    r, c = np.arange(N)[:, None], np.arange(K // 32)[None]
    byte = rng.integers(40, 200, (N, 1)) + rng.integers(-6, 7, (N, K // 32))
    flat[((r // 128) * 4 + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4] = byte
    x = torch.randn(3, K, device=DEV) * torch.tensor([1e-30, 1.0, 1e10], device=DEV)[:, None]
    x = x.to(torch.bfloat16)
    y = fl.mxfp4_matvec(x, u8(codes), u8(flat))
    W = ref.weight(codes, flat, "mxfp4")
    want, mag = ref.f64(x) @ W.T, np.abs(ref.f64(x)) @ np.abs(W).T
    got = ref.f64(y)
    ok = (np.abs(want) < 1e38) & (mag > 1e-30)
    within(got[ok], want[ok], ((K + 8) * F32 * mag * (1 + BF16) + BF16 * np.abs(want))[ok], "far scales")
    w = weight(64, 256, "nvfp4", 0)
    x = torch.randn(4, 256, device=DEV).to(torch.bfloat16)
    good = fl.weight_only_linear(x, w)
    x[1, 3], x[2, 200] = float("nan"), float("inf")
    y = fl.weight_only_linear(x, w)
    assert torch.equal(y[0], good[0]) and torch.equal(y[3], good[3])
    assert y[1].isnan().all() and not y[2].isfinite().any()
    status_ok()


def test_matvec_out_strides_and_refusals():
    w = weight(70, 128, "nvfp4", 0)
    base = torch.randn(5, 304, device=DEV).to(torch.bfloat16)
    x = base[:, 8:136]
    room = torch.full((5, 101), 7.0, device=DEV, dtype=torch.bfloat16)
    y = fl.weight_only_linear(x, w, out=room[:, 3:73])
    assert torch.equal(y, fl.weight_only_linear(x.contiguous(), w))
    assert (room[:, :3] == 7).all() and (room[:, 73:] == 7).all()
    with pytest.raises(ValueError, match="holds"):
        fl.nvfp4_matvec(x, w.codes, w.scales[:512], w.g)  # 128 x 8 scales take 1024 bytes
    with pytest.raises(ValueError, match="values a row"):
        fl.nvfp4_matvec(base[:, :64], w.codes, w.scales, w.g)
    with pytest.raises(TypeError, match="uint8"):
        fl.nvfp4_matvec(x, w.codes, w.scales, w.g, x_scales=w.scales)
    with pytest.raises(fl.Fp4LinError, match="UNSUPPORTED"):
        fl.nvfp4_matvec(base.repeat(4, 1)[:, :128], w.codes, w.scales, w.g)
    status_ok()


# ------------------------------------------------------------------ tables
def table_case(B, P, width, seed, new_top=40):
    rng = np.random.default_rng(seed)
    rows = width * P
    lens = rng.integers(0, rows // 2 + 1, B)
    new = np.where(rng.random(B) < 0.3, 0, rng.integers(1, min(new_top, rows // 2) + 1, B))
    had, need = -(-lens // P), -(-(lens + new) // P)
    ids = rng.permutation(int(need.sum()) + 4)
    table = rng.integers(-9, -1, (B, width))
    k = 0
    for b in range(B):
        table[b, :had[b]] = ids[k:k + had[b]]
        k += had[b]
    return lens, new, table, np.concatenate([[-5, -5], ids[k:]])


@pytest.mark.parametrize("B,P,width", [(1, 16, 4), (3, 64, 2), (40, 32, 9), (513, 16, 12), (1025, 128, 3), (8192, 16, 5)])
def test_tables(B, P, width):
    lens, new, table, free = table_case(B, P, width, B)
    if B == 3:
        lens[:], new[:] = [0, P, P - 1], [0, 1, 1]
    for most in (int(new.sum()) or 1, int(new.sum()) + 77):
        t = gpu(np.pad(table, ((0, 0), (0, 3)), constant_values=-77))
        cu, slots, head = fl.kv_block_tables(t[:, :width], gpu(lens), gpu(new), gpu(free), gpu([2]), P, max_tokens=most)
        status_ok()
        wt, wcu, ws, wh = ref.tables(table, lens, new, free, 2, P, most)
        assert np.array_equal(t[:, :width].cpu(), wt) and (t[:, width:] == -77).all()
        assert np.array_equal(cu.cpu(), wcu) and np.array_equal(slots.cpu(), ws) and head.item() == wh


def test_tables_report_what_does_not_fit():
    P = 16
    table = np.full((4, 2), -3)
    table[1, 0] = 6

    def call(lens, new, free, most, head=0):
        t = gpu(table)
        cu, slots, nh = fl.kv_block_tables(t, gpu(lens), gpu(new), gpu(free), gpu([head]), P, max_tokens=most)
        return t.cpu().numpy(), cu.tolist(), slots.tolist(), nh.item(), fl.device_status()

    ok = ([0, 3, 0, 0], [1, 2, 0, 17], [8, 9, 10, 11])
    t, cu, slots, nh, st = call(*ok, 20)
    assert st == 0 and cu == [0, 1, 3, 3, 20] and nh == 3
    assert slots == [128, 99, 100] + [144 + i for i in range(16)] + [160]
    # the free list runs out: the last page is missing
    t, cu, slots, nh, st = call(ok[0], ok[1], [8, 9], 20)
    assert st == OUT_OF_RANGE and nh == 2 and t[3].tolist() == [9, -1] and slots[-1] == -1 and slots[3] == 144
    # fewer slots than tokens
    t, cu, slots, nh, st = call(*ok, 2)
    assert st == OUT_OF_RANGE and cu == [0, 1, 2, 2, 2] and slots == [128, 99]
    # a negative length gets nothing, the others their own
    t, cu, slots, nh, st = call([0, 3, -1, 0], [1, 2, 5, 1], [8, 9, 10, 11], 6)
    assert st == OUT_OF_RANGE and cu == [0, 1, 3, 3, 4] and slots == [128, 99, 100, 144, -1, -1]
    # more rows than the table's width
    t, cu, slots, nh, st = call([0, 3, 0, 31], [1, 2, 0, 3], [8, 9, 10, 11], 6)
    assert st == OUT_OF_RANGE and nh == 1 and slots == [128, 99, 100, -1, -1, -1]
    # a head outside the list
    t, cu, slots, nh, st = call(*ok, 20, head=5)
    assert st == OUT_OF_RANGE and nh == 5 and slots[0] == -1 and slots[1] == 99
    # lengths that no 32-bit sum holds
    big = 2 ** 31 - 1
    t, cu, slots, nh, st = call([big] * 4, [big] * 4, [8, 9, 10, 11], 5)
    assert st == OUT_OF_RANGE and slots == [-1] * 5 and cu == [0, 5, 5, 5, 5] and (t == table).all()
    with pytest.raises(ValueError, match="at least 1"):
        fl.kv_block_tables(gpu(table), *[gpu([0] * 4)] * 2, gpu([1]), gpu([0]), P, max_tokens=0)
    h = gpu([0])
    with pytest.raises(fl.Fp4LinError, match="INVALID"):
        fl.kv_block_tables(gpu(table), *[gpu([0] * 4)] * 2, gpu([1]), h, P, max_tokens=1, next_head=h)


# ------------------------------------------------------------------ append
def fresh_cache(NP, H, P, D, seed):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (NP, H, P, D), dtype=np.uint8)
    byte = rng.integers(110, 130, (NP, H), dtype=np.uint8)
    return codes, byte


def check_append(k, v, slots, kc, kb, vc, vb, P):
    """Run the GPU call and the plain form on copies; both caches bit for bit."""
    gk, gkb, gv, gvb = u8(kc), u8(kb), u8(vc), u8(vb)
    fl.kv_fp8_store(k, v, gpu(slots), (gk, gkb), (gv, gvb))
    for x, c, b, gc, gb in ((k, kc, kb, gk, gkb), (v, vc, vb, gv, gvb)):
        ref.append(ref.f64(x), list(slots), c, b, P)
        assert np.array_equal(gb.cpu().numpy(), b), "scales"
        got = gc.cpu().numpy()
        same = (got == c) | (np.isnan(ref.E4M3[got]) & np.isnan(ref.E4M3[c]))
        assert same.all(), f"codes differ at {np.argwhere(~same)[:4].tolist()}"


@pytest.mark.parametrize("H,P,D,runs", [
    (1, 16, 64, [(0, 0, 1)]), (2, 16, 128, [(3, 5, 1), (0, 15, 1), (1, 0, 16)]), (3, 64, 128, [(2, 10, 50), (0, 0, 64), (1, 63, 1)]),
    (2, 128, 64, [(1, 0, 128), (0, 127, 1), (2, 1, 126)]), (8, 128, 128, [(0, 0, 128), (3, 3, 100)]),
    (5, 32, 64, [(i, (7 * i) % 32, 1) for i in range(60)]), (1, 16, 128, [(i, 0, 16) for i in range(200)])])
def test_append(H, P, D, runs):
    NP = max(p for p, _, _ in runs) + 2
    slots = np.concatenate([p * P + r + np.arange(n) for p, r, n in runs] + [[-1, -1]])
    g = torch.Generator().manual_seed(H * P + D)
    T = len(slots)
    kv = (torch.randn(T, 2, H, D, generator=g) * torch.exp2(torch.randn(T, 1, H, 1, generator=g) * 4)).to(torch.bfloat16)
    kv[-2:] = float("nan")  # rows of slot -1 are not read
    kv = kv.to(DEV)
    kc, kb = fresh_cache(NP, H, P, D, 1)
    vc, vb = fresh_cache(NP, H, P, D, 2)
    check_append(kv[:, 0], kv[:, 1], slots, kc, kb, vc, vb, P)
    status_ok()


def test_append_token_by_token_as_values_grow_and_shrink():
    H, P, D = 2, 16, 64
    kc, kb = fresh_cache(2, H, P, D, 5)
    vc, vb = fresh_cache(2, H, P, D, 6)
    g = torch.Generator().manual_seed(1)
    for t in range(P):
        x = (torch.randn(1, 2, H, D, generator=g) * 2.0 ** [0, -3, 5, 40, 39, -60, 41, 60, 0, 80, 99, 100, 90, 1, 2, 3][t])
        x = x.to(torch.bfloat16).to(DEV)
        check_append(x[:, 0], x[:, 1], [P + t], kc, kb, vc, vb, P)
    status_ok()


def test_append_zeros_infinities_nan_and_tiny_values():
    H, P, D = 1, 16, 64
    kc, kb = fresh_cache(3, H, P, D, 5)
    vc, vb = fresh_cache(3, H, P, D, 6)
    x = torch.randn(4, H, D).to(torch.bfloat16)
    x[0, 0, 1], x[0, 0, 2], x[0, 0, 3] = float("inf"), float("-inf"), float("nan")
    x[1] = 0
    x[2] = x[2].float() * 1e-39
    x[3] = 3.0e38
    for rows, slots in ((x[0:1], [0]), (x[1:2], [16]), (x[2:3], [32]), (x[1:2], [17]), (x[2:3], [18]), (x[3:4], [33])):
        d = rows.to(DEV)
        check_append(d, d, slots, kc, kb, vc, vb, P)
    status_ok()


def test_append_bad_slots_and_strides():
    H, P, D, NP = 2, 16, 128, 4
    kc, kb = fresh_cache(NP, H, P, D, 5)
    vc, vb = fresh_cache(NP, H, P, D, 6)
    x = torch.randn(5, 3 * H * D + 8, device=DEV).to(torch.bfloat16)  # slices of one projection's output
    k, v = x[:, :H * D].view(5, H, D), x[:, H * D:2 * H * D].view(5, H, D)
    check_append(k, v, [64, 17, -1, -2, 2 ** 31 - 1], kc, kb, vc, vb, P)
    assert fl.device_status() == OUT_OF_RANGE
    with pytest.raises(ValueError, match="contiguous rows"):
        fl.kv_fp8_store(x[:, :2 * H * D].view(5, H, 2 * D)[:, :, :D], v, gpu([0] * 5), (u8(kc), u8(kb)), (u8(vc), u8(vb)))
    with pytest.raises(ValueError, match=r"must be \[5, 2, 128\]"):
        fl.kv_fp8_store(k[:4], v, gpu([0] * 5), (u8(kc), u8(kb)), (u8(vc), u8(vb)))
    with pytest.raises(ValueError, match="same shape"):
        fl.kv_fp8_store(k, v, gpu([0] * 5), (u8(kc), u8(kb)), (u8(vc[1:]), u8(vb[1:])))


# ------------------------------------------------------------------ attention
def attention_case(B, H, G, D, P, lens, new, seed=0, sigma=2.0, spread=1.0):
    """A cache with pages in a random order whose rows behind each request's last are NaN codes."""
    rng = np.random.default_rng(seed)
    lens, new = np.asarray(lens), np.asarray(new)
    need = -(-(lens + new) // P)
    width, NP = int(max(need.max(), 1)) + 1, int(need.sum()) + 2
    ids = rng.permutation(NP)
    table = np.full((B, width), -1)
    k = 0
    for b in range(B):
        table[b, :need[b]] = ids[k:k + need[b]]
        k += need[b]
    caches = []
    for _ in range(2):
        x = rng.standard_normal((NP, H, P, D)) * 2.0 ** (spread * rng.standard_normal((NP, H, 1, 1)))
        byte = ref.block_byte(np.abs(x).max((2, 3)))
        codes = ref.e4m3_bytes(x * 2.0 ** (127.0 - byte)[..., None, None])
        for b in range(B):
            if need[b] and (lens[b] + new[b]) % P:
                codes[table[b, need[b] - 1], :, (lens[b] + new[b]) % P:] = 0x7F
        caches.append((codes, byte.astype(np.uint8)))
    T = int(new.sum()) + 3
    q = torch.tensor(rng.standard_normal((T, H * G, D)) * sigma).to(torch.bfloat16)
    return q, caches, table, lens, np.concatenate([[0], np.cumsum(new)])


def attention_check(q, caches, table, lens, cu, P, scale=None, max_new=None, max_len=None, strided=False):
    (kc, kb), (vc, vb) = caches
    T, HQ, D = q.shape
    n = np.diff(cu)
    max_new = int(max(n.max(), 1)) if max_new is None else max_new
    max_len = int(max((lens + n).max(), 1)) if max_len is None else max_len
    qd = q.to(DEV)
    if strided:  # a slice of a wider projection
        room = torch.full((T, HQ * D + 72), float("nan"), dtype=torch.bfloat16, device=DEV)
        room[:, 8:8 + HQ * D] = qd.reshape(T, HQ * D)
        qd = room[:, 8:8 + HQ * D].view(T, HQ, D)
    out = torch.full((T, HQ, D), 123.0, dtype=torch.bfloat16, device=DEV)
    fl.kv_fp8_attention(qd, (u8(kc), u8(kb)), (u8(vc), u8(vb)), gpu(table), gpu(lens), gpu(cu), max_new=max_new,
                        max_len=max_len, scale=scale, out=out)
    got = ref.f64(out)
    want, spread, dots = ref.attention(ref.f64(q), kc, kb, vc, vb, table, lens, cu, P, D ** -0.5 if scale is None else scale)
    mine = ~np.isnan(want)
    assert (got[~mine] == 123.0).all(), "rows of no request were written"
    # a weight's relative error: its score's (binary32 dot of D terms and two scalings, q's f16
    # rounding where it is below 2^-14 of its row, the exponential's 2^-22), twice for numerator and
    # denominator; its own rounding to f16 (2^-11, and 2^-25 absolute of the largest weight, which
    # meets at most all of sum |v|); binary32 sums over the keys
    L = int((lens + n).max())
    w = 2 * ((D + 6) * F32 * dots + 2.0 ** -21) + F16 + 2 * L * F32
    tol = w * spread
    within(got[mine], want[mine], (tol * (1 + BF16) + BF16 * np.abs(want) + 2.0 ** -25 * 0)[mine], "attention")
    return out


@pytest.mark.parametrize("B,H,G,D,P,lens,new", [
    (1, 1, 1, 64, 16, [0], [1]),
    (1, 1, 1, 128, 16, [5], [1]),
    (3, 2, 4, 128, 16, [0, 15, 16], [1, 1, 1]),
    (4, 2, 8, 64, 32, [100, 0, 31, 7], [1, 0, 1, 1]),
    (2, 3, 5, 128, 64, [200, 63], [1, 1]),
    (2, 1, 16, 128, 128, [300, 127], [1, 1]),
    (3, 2, 3, 64, 16, [40, 0, 33], [4, 5, 0]),
    (2, 2, 2, 128, 32, [130, 0], [8, 3]),
    (1, 1, 1, 128, 16, [3000], [1]),
    (5, 1, 4, 128, 64, [2500, 1, 128, 0, 1023], [2, 1, 2, 2, 1]),
    (2, 2, 4, 128, 64, [37, 0], [33, 64]),
    (1, 1, 8, 64, 16, [0], [70]),
    (3, 1, 3, 128, 16, [129, 5, 0], [131, 1, 60]),
    (1, 2, 16, 128, 32, [300], [41]),
    (2, 1, 1, 64, 128, [500, 0], [200, 257])])
def test_attention(B, H, G, D, P, lens, new):
    attention_check(*attention_case(B, H, G, D, P, lens, new, seed=B + G + D + P), P)
    status_ok()


def test_attention_larger_bounds_strides_and_scale():
    q, caches, table, lens, cu = attention_case(3, 2, 4, 128, 32, [70, 200, 3], [2, 1, 2], seed=9)
    table = np.pad(table, ((0, 0), (0, 80)), constant_values=-1)
    attention_check(q, caches, table, lens, cu, 32, max_new=2, max_len=2000, strided=True)
    attention_check(q, caches, table, lens, cu, 32, max_new=50, max_len=300, scale=0.3)
    attention_check(q, caches, table, lens, cu, 32, scale=-0.05)
    attention_check(q, caches, table, lens, cu, 32, scale=0.0)
    status_ok()


@pytest.mark.parametrize("new", [1, 90])
def test_attention_page_scales_far_apart_and_zero_pages(new):
    q, ((kc, kb), (vc, vb)), table, lens, cu = attention_case(2, 2, 4, 128, 16, [400, 30], [new, new], seed=4, spread=3.0)
    vc[table[0, 1]] = 0  # a page of zero values, at its scale and at byte 0
    vc[table[0, 3]] = 0
    vb[table[0, 3]] = 0
    vc[table[0, 0]], vb[table[0, 0]] = 0, 0
    kc[table[0, 2]], kb[table[0, 2]] = 0, 0
    attention_check(q, ((kc, kb), (vc, vb)), table, lens, cu, 16)
    vc[:], vb[:] = 0, 0  # nothing but zeros: the answer is zero
    attention_check(q, ((kc, kb), (vc, vb)), table, lens, cu, 16)
    status_ok()


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("q_scale,v_shift", [(2.0 ** -100, 0), (2.0 ** 60, 0), (1.0, 60), (1.0, -60)])
def test_attention_extreme_magnitudes(new, q_scale, v_shift):
    q, ((kc, kb), (vc, vb)), table, lens, cu = attention_case(1, 1, 4, 64, 32, [170], [new], seed=4)
    kb = (kb.astype(int) - int(np.log2(q_scale))).astype(np.uint8)  # q and k undo each other
    vb = (vb.astype(int) + v_shift).astype(np.uint8)
    attention_check((q.float() * q_scale).to(torch.bfloat16), ((kc, kb), (vc, vb)), table, lens, cu, 32)
    status_ok()


@pytest.mark.parametrize("G,new", [(2, 5), (4, 60), (1, 300)])
def test_attention_nan_values_reach_only_the_rows_that_see_them(G, new):
    q, ((kc, kb), (vc, vb)), table, lens, cu = attention_case(2, 2, G, 64, 32, [70, 0], [new, new], seed=11)
    for b, p, h, d in ((0, 70 + new // 2, 1, 9), (0, 71, 0, 63), (1, new - 1, 1, 0)):
        vc[table[b, p // 32], h, p % 32, d] = 0xFF if d else 0x7F
    out = torch.zeros(q.shape, dtype=torch.bfloat16, device=DEV)
    fl.kv_fp8_attention(q.to(DEV), (u8(kc), u8(kb)), (u8(vc), u8(vb)), gpu(table), gpu(lens), gpu(cu), max_new=new,
                        max_len=70 + new, out=out)
    status_ok()
    got, want = ref.f64(out), ref.attention(ref.f64(q), kc, kb, vc, vb, table, lens, cu, 32, 0.125)[0]
    # the reference gives every key that a row does not see no part in it
    assert np.array_equal(np.isnan(got[:2 * new]), np.isnan(want[:2 * new]))
    ok = ~np.isnan(want)
    assert np.abs(got[ok] - want[ok]).max() < 0.05


@pytest.mark.parametrize("L", [100, 129, 900, 1024, 1100, 2048, 2300, 20000])
def test_attention_split_counts(L):
    """One split, the cluster's two to eight, and the workspace's many."""
    attention_check(*attention_case(2, 1, 4, 64, 32, [L - 1, L // 3], [1, 1], seed=L), 32)
    status_ok()


@pytest.mark.parametrize("B,H,G,D,P,lens,new,max_len", [
    (1, 2, 8, 128, 64, [2046], [4], None),             # the last key of a block
    (1, 1, 8, 64, 16, [2047], [5], None),              # and a block more, with four keys in it
    (2, 1, 4, 128, 32, [5000, 40], [70, 5], None),     # requests of fewer splits, and of one
    (2, 1, 4, 64, 128, [2900, 3100], [100, 3], 9000),  # splits that no request reaches; a tile of 144 rows
    (3, 1, 8, 128, 64, [6000, 6100, 0], [40, 1, 0], None),  # beside a single token's split kernel and its merge
    (1, 1, 1, 64, 16, [0], [2500], None)])             # rows whose first split has keys and whose later ones none
def test_attention_many_rows_with_the_keys_split(B, H, G, D, P, lens, new, max_len):
    q, caches, table, lens, cu = attention_case(B, H, G, D, P, lens, new, seed=H + G + D + P)
    table = np.pad(table, ((0, 0), (0, max(0, (max_len or 0) // P + 1 - table.shape[1]))), constant_values=-1)
    attention_check(q, caches, table, lens, cu, P, max_len=max_len)
    status_ok()


def test_attention_prompts_among_many_decoding_requests():
    """More than a thread's one request in the plan; tiles alone and, at the end, shared."""
    lens, new = np.full(1500, 3), np.ones(1500, int)
    lens[7::100] = 40
    new[[3, 700, 701, 1499]] = [130, 70, 0, 300]
    lens[[700, 1499]] = 600, 900
    attention_check(*attention_case(1500, 1, 2, 64, 16, lens, new, seed=3), 16)
    status_ok()
    # more tiles than SMs, ends of requests inside a tile
    attention_check(*attention_case(3, 10, 16, 64, 64, [30, 600, 5], [83, 90, 81], seed=4), 64)
    status_ok()


def test_attention_few_long_requests_where_the_batch_allows_more():
    """98 requests of many rows, three CTAs each, in a batch that might have had 150."""
    lens, new = np.full(150, 1600), np.ones(150, int)
    new[:98] = 26
    q, caches, table, lens, cu = attention_case(150, 1, 1, 64, 128, lens, new, seed=6)
    attention_check(q, caches, table, lens, cu, 128)
    # fewer than its workspace has room for: 140 requests of q's length
    n = np.where(np.arange(150) < 90, 26, 0)
    cu = np.concatenate([[0], np.cumsum(n)])
    attention_check(q[:cu[-1]], caches, table, lens, cu, 128)
    status_ok()


def test_attention_offsets_that_fall_and_rise_with_long_requests():
    """Overlapping requests, which no plan has room for: reported, and nothing but rows of q's is written."""
    q, caches, table, lens, cu = attention_case(9, 1, 4, 64, 16, [700] * 9, [60] * 9, seed=5)
    (kc, kb), (vc, vb) = caches
    cu = np.array([0, 60, 0, 60, 0, 60, 0, 60, 0, 60])
    room = torch.full((80, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    fl.kv_fp8_attention(q[:60].to(DEV), (u8(kc), u8(kb)), (u8(vc), u8(vb)), gpu(table), gpu(lens), gpu(cu), max_new=60,
                        max_len=760, out=room[:60])
    assert fl.device_status() == OUT_OF_RANGE and (room[60:] == 7).all()


def test_attention_nan_values_and_missing_pages_where_the_keys_are_split():
    q, caches, table, lens, cu = attention_case(1, 1, 8, 64, 16, [4000], [60], seed=4)
    (kc, kb), (vc, vb) = caches
    vc[table[0, 5], 0, 3, 7] = 0x7F                  # a key that all rows see
    vc[table[0, 4030 // 16], 0, 4030 % 16, 9] = 0xFF  # one that the last 30 tokens see
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
    a = [(u8(kc), u8(kb)), (u8(vc), u8(vb)), gpu(table), gpu(lens), gpu(cu)]
    fl.kv_fp8_attention(q.to(DEV), *a, max_new=60, max_len=4060, out=out)
    got = torch.isnan(out[:60]).cpu()
    want = torch.zeros_like(got)
    want[:, :, 7] = True
    want[30:, :, 9] = True
    assert torch.equal(got, want)
    status_ok()
    table[0, 128:] = -1  # whole splits without a page
    a[2] = gpu(table)
    fl.kv_fp8_attention(q.to(DEV), *a, max_new=60, max_len=4060, out=out)
    assert fl.device_status() == OUT_OF_RANGE
    t64 = ref.attention(ref.f64(q), kc, kb, vc, vb, table, lens, cu, 16, 64 ** -0.5)[0][:60]
    have = ~np.isnan(t64)
    assert np.abs(ref.f64(out)[:60][have] - t64[have]).max() < 0.05
    assert torch.isnan(out[:60, :, 7]).all() and not torch.isnan(out[:60, :, 8:]).any()


def test_attention_many_rows_over_and_over():
    """Short and long contexts back to back, each with the same bits every time: no wait depends on luck."""
    for D, lens, new in ((64, [0, 100, 300, 0], [300, 40, 256, 33]), (128, [60, 1000, 0, 129], [129, 300, 64, 512])):
        q, caches, table, lens, cu = attention_case(4, 2, 2, D, 32, lens, new, seed=D)
        (kc, kb), (vc, vb) = caches
        a = [q.to(DEV), (u8(kc), u8(kb)), (u8(vc), u8(vb)), gpu(table), gpu(lens), gpu(cu)]
        kw = dict(max_new=max(new), max_len=int((lens + np.asarray(new)).max()))
        first = fl.kv_fp8_attention(*a, **kw)
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        T = int(cu[-1])
        same = torch.ones((), dtype=torch.bool, device=DEV)
        for k in range(400):
            out = fl.kv_fp8_attention(*a, **kw)
            fl.kv_fp8_attention(*a, **kw, stream=other)  # and beside itself
            same &= (out[:T].view(torch.int16) == first[:T].view(torch.int16)).all()
        torch.cuda.synchronize()
        assert bool(same)
        status_ok()


def test_attention_skips_and_reports_what_breaks_its_bounds():
    q, caches, table, lens, cu = attention_case(3, 1, 2, 64, 16, [20, 40, 3], [2, 3, 1], seed=2)
    (kc, kb), (vc, vb) = caches

    def call(table=table, lens=lens, cu=cu, max_new=3, max_len=43, **kw):
        out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=DEV)
        fl.kv_fp8_attention(q.to(DEV), (u8(kc), u8(kb)), (u8(vc), u8(vb)), gpu(table), gpu(lens), gpu(cu),
                            max_new=max_new, max_len=max_len, out=out, **kw)
        return out, fl.device_status()

    good, st = call()
    assert st == 0
    # request 1 has more new tokens, or more rows, than the host said: skipped, the others not
    for kw in (dict(max_new=2), dict(max_len=42), dict(lens=np.array([20, -1, 3]))):
        out, st = call(**kw)
        assert st == OUT_OF_RANGE and (out[2:5] == 5).all()
        assert torch.equal(out[:2], good[:2]) and torch.equal(out[5:], good[5:])
    # offsets that fall, or pass the rows of q
    out, st = call(cu=np.array([0, 2, 1, 2]))
    assert st == OUT_OF_RANGE and torch.equal(out[:1], good[:1]) and (out[2:] == 5).all()
    out, st = call(cu=np.array([0, 2, 5, 2 ** 31 - 1]))
    assert st == OUT_OF_RANGE and (out[5:] == 5).all() and torch.equal(out[:5], good[:5])
    # a page that is none counts as not there
    for bad in (-1, len(kb), 2 ** 31 - 1):
        t = table.copy()
        t[1, 1] = bad
        out, st = call(table=t)
        assert st == OUT_OF_RANGE
        want = ref.attention(ref.f64(q), kc, kb, vc, vb, np.where(t >= len(kb), -1, t), lens, cu, 16, 64 ** -0.5)[0]
        live = ~np.isnan(want)
        assert np.abs(ref.f64(out)[live] - want[live]).max() < 0.05
        assert torch.equal(out[:2], good[:2])
    t = table.copy()
    t[2] = -1  # no page at all: nothing to see, the row is zero
    out, st = call(table=t)
    assert st == OUT_OF_RANGE and (out[5] == 0).all() and (out[6:] == 5).all()


def test_attention_refusals():
    q, ((kc, kb), (vc, vb)), table, lens, cu = attention_case(1, 2, 2, 64, 16, [3000], [1])
    a = [q.to(DEV), (u8(kc), u8(kb)), (u8(vc), u8(vb)), gpu(table), gpu(lens), gpu(cu)]
    with pytest.raises(fl.Fp4LinError, match="INVALID"):
        fl.kv_fp8_attention(*a, max_new=1, max_len=table.shape[1] * 16 + 1)
    with pytest.raises(fl.Fp4LinError, match="WORKSPACE"):
        wide = gpu(np.pad(table, ((0, 0), (0, 1400)), constant_values=-1))  # more than a cluster's splits
        fl.kv_fp8_attention(*a[:3], wide, *a[4:], max_new=1, max_len=20000, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(fl.Fp4LinError, match="WORKSPACE"):  # many rows, whose keys may be shared
        fl.kv_fp8_attention(*a, max_new=20, max_len=3001, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="a multiple of 2 heads"):
        fl.kv_fp8_attention(a[0][:, :3], *a[1:], max_new=1, max_len=3001)
    with pytest.raises(TypeError, match="pair"):
        fl.kv_fp8_attention(a[0], a[1][0][0], *a[2:], max_new=1, max_len=3001)
    with pytest.raises(TypeError, match="lens must be torch.int32"):
        fl.kv_fp8_attention(*a[:4], a[4].long(), a[5], max_new=1, max_len=3001)
    status_ok()


# ------------------------------------------------------------------ a serving step
class Step:
    """One layer's step for a batch: norm, q/k/v product, tables, append, attention, output product."""

    def __init__(self, B, H, G, D, P, model, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        self.B, self.H, self.G, self.D, self.P, self.model = B, H, G, D, P, model
        self.norm = (1 + 0.1 * rnd(model)).to(torch.bfloat16)
        self.qkv = fl.prepare_weight((rnd((G + 2) * H * D, model) / model ** 0.5).to(torch.bfloat16), "nvfp4", 16)
        self.o = fl.prepare_weight((rnd(model, G * H * D) / (G * H * D) ** 0.5).to(torch.bfloat16), "mxfp4", 32)
        NP, width = 4 * B, 4
        self.k = (torch.full((NP, H, P, D), 0x7F, dtype=torch.uint8, device=DEV), torch.zeros(NP, H, dtype=torch.uint8, device=DEV))
        self.v = (torch.full((NP, H, P, D), 0x7F, dtype=torch.uint8, device=DEV), torch.zeros(NP, H, dtype=torch.uint8, device=DEV))
        self.table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        self.free = torch.arange(NP, dtype=torch.int32, device=DEV).flip(0).contiguous()
        self.lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.head = torch.zeros(1, dtype=torch.int32, device=DEV)

    def __call__(self, x, residual, new, max_new, stream=None):
        T, HD = x.shape[0], self.H * self.D
        kw = dict(stream=stream)
        c, s, residual = fl.rmsnorm_mxfp8(x, self.norm, residual, hadamard=16, **kw)
        y = fl.weight_only_linear(c, self.qkv, x_scales=s, **kw)
        q, k, v = (t.view(T, -1, self.D) for t in y.split([self.G * HD, HD, HD], 1))
        cu, slots, head = fl.kv_block_tables(self.table, self.lens, new, self.free, self.head, self.P, max_tokens=T, **kw)
        fl.kv_fp8_store(k, v, slots, self.k, self.v, **kw)
        a = fl.kv_fp8_attention(q, self.k, self.v, self.table, self.lens, cu, max_new=max_new, max_len=4 * self.P, **kw)
        out = fl.weight_only_linear(a.view(T, -1), self.o, **kw)
        return out, residual, y, a, head

    def advance(self, new, head):
        self.lens += new
        self.head.copy_(head)


def test_serving_steps_against_the_plain_forms():
    """Prompts of different lengths, then single tokens, through every operator in turn; keys and
    values as the caches hold them are checked by the append's own tests, here the whole chain."""
    st = Step(3, 2, 2, 64, 16, 256)
    g = torch.Generator(device=DEV).manual_seed(5)
    past = [[], [], []]  # the k and v rows of each request, as the products gave them
    for new in ([7, 3, 5], [1, 1, 1], [1, 0, 1], [10, 1, 3], [1, 1, 1]):
        T = sum(new)
        x = torch.randn(T, 256, generator=g, device=DEV).to(torch.bfloat16)
        r = torch.randn(T, 256, generator=g, device=DEV).to(torch.bfloat16)
        n = gpu(new)
        out, residual, y, a, head = st(x, r, n, max(new))
        status_ok()
        kc, kb, vc, vb = (t.cpu().numpy() for t in (*st.k, *st.v))
        q, k, v = (t.reshape(T, -1, 64) for t in np.split(ref.f64(y), [256, 384], 1))
        cu, lens, table = np.concatenate([[0], np.cumsum(new)]), st.lens.cpu().numpy(), st.table.cpu().numpy()
        want, spread, dots = ref.attention(q, kc, kb, vc, vb, table, lens, cu, 16, 64 ** -0.5)
        L = int((lens + new).max())
        tol = (2 * (70 * F32 * dots + 2.0 ** -21) + F16 + 2 * L * F32) * spread * (1 + BF16) + BF16 * np.abs(want)
        within(ref.f64(a), want, tol, "attention in the chain")
        for b in range(3):  # the caches hold what was appended, within E4M3's step of the page's scale
            past[b] += [(k[t], v[t]) for t in range(cu[b], cu[b + 1])]
            for p, (kk, vv) in enumerate(past[b]):
                for x64, codes, byte in ((kk, kc, kb), (vv, vc, vb)):
                    page, row = table[b, p // 16], p % 16
                    step = 2.0 ** (byte[page].astype(float) - 127)[:, None]
                    # once when written and once each time the page's exponent grew: subnormals only
                    within(ref.E4M3[codes[page, :, row]] * step, x64, 2.0 ** -4 * np.abs(x64) + 4 * 2.0 ** -10 * step, "cache")
        matvec_rotated_check(out, a.view(T, -1), st.o, 32)
        st.advance(n, head)


def test_memory_made_for_another_stream_is_not_taken_from_pending_work():
    """Memory that the current stream has freed but not finished with is given to no call on another."""
    q, caches, table, lens, cu = attention_case(2, 1, 4, 64, 32, [300, 100], [40, 30], seed=1)
    a = [q.to(DEV), *[(u8(c), u8(b)) for c, b in caches], gpu(table), gpu(lens), gpu(cu)]
    want = fl.kv_fp8_attention(*a, max_new=40, max_len=340).clone()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(3):
        held = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device=DEV)
        seen = torch.empty_like(held)
        torch.cuda._sleep(20_000_000)
        seen.copy_(held)
        del held
        out = fl.kv_fp8_attention(*a, max_new=40, max_len=340, stream=other)
        torch.cuda.synchronize()
        assert (seen == 3).all() and torch.equal(out[:70], want[:70])
        del out, seen
    status_ok()


def test_serving_step_captured_replayed_and_on_another_stream():
    runs = []
    for mode in ("eager", "graph", "stream"):
        st = Step(4, 2, 4, 128, 16, 256, seed=3)
        g = torch.Generator(device=DEV).manual_seed(8)
        xs = [(torch.randn(4, 256, generator=g, device=DEV).to(torch.bfloat16),
               torch.randn(4, 256, generator=g, device=DEV).to(torch.bfloat16)) for _ in range(20)]
        new = torch.ones(4, dtype=torch.int32, device=DEV)
        x, r = xs[0][0].clone(), xs[0][1].clone()
        got = []
        if mode == "graph":
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out, res, _, _, head = st(x, r, new, 1)
                st.advance(new, head)
            for a, b in xs:
                x.copy_(a)
                r.copy_(b)
                graph.replay()
                got.append((out.clone(), res.clone()))
        elif mode == "stream":
            side = torch.cuda.Stream()
            for a, b in xs:
                side.wait_stream(torch.cuda.current_stream())
                out, res, _, _, head = st(a, b, new, 1, stream=side)
                torch.empty(1 << 20, device=DEV).fill_(float("nan"))  # takes freed memory, if it is given out
                torch.cuda.current_stream().wait_stream(side)
                st.advance(new, head)
                got.append((out.clone(), res.clone()))
        else:
            for a, b in xs:
                out, res, _, _, head = st(a, b, new, 1)
                st.advance(new, head)
                got.append((out, res))
        status_ok()
        runs.append((got, st))
    (eager, s0), *others = runs
    for got, s in others:
        for (o0, r0), (o1, r1) in zip(eager, got):
            assert torch.equal(o0, o1) and torch.equal(r0, r1)
        assert torch.equal(s0.table, s.table) and torch.equal(s0.lens, s.lens)
        for a, b in zip((*s0.k, *s0.v), (*s.k, *s.v)):
            assert torch.equal(a, b)
