"""The serving operators without a GPU: exports, the host-side refusals of the C ABI (fake device
pointers are never dereferenced) and of the binding, and the reference forms the GPU tests use."""
import os
import re

import numpy as np
import pytest
import torch

import mxfp4_microscaled_bit_b200 as fl
import serving_ref as ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fp4lin_serving.h")
INVALID, SHAPE, MISALIGNED = 1, 2, 3
P = 0x10000  # 16-byte aligned, never dereferenced on these paths


def test_every_declared_symbol_is_exported():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(\w+)\s*\(", src, flags=re.M))
    assert names == set(fl.SERVING_EXPORTS) and not names & set(fl.EXPORTS)
    for n in names:
        assert hasattr(fl.lib(), n), n


def test_norm_refusals():
    def f(x=P, ldx=64, r=P, ldr=64, w=P, eps=1e-6, had=0, rows=4, cols=64, c=P, s=P, out=P, lds=64):
        return fl.lib().rmsnorm_mxfp8(x, ldx, r, ldr, w, eps, had, rows, cols, c, s, out, lds, None)

    for kw in (dict(x=None), dict(w=None), dict(c=None), dict(s=None), dict(r=None), dict(out=None), dict(rows=0),
               dict(cols=0), dict(ldx=32), dict(ldr=32), dict(lds=32), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(had=8)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(cols=48), dict(ldx=68), dict(ldr=68), dict(lds=68), dict(cols=32800, ldx=32800, ldr=32800, lds=32800)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=P + 8), dict(w=P + 2), dict(c=P + 1), dict(s=P + 4), dict(out=P + 8), dict(r=P + 8)):
        assert f(**kw) == MISALIGNED, kw


@pytest.mark.parametrize("nv", [True, False])
def test_matvec_refusals(nv):
    def f(x=P, xs=None, M=4, K=128, ldx=128, had=0, w=P, ws=P, g=P, y=P, N=10, ldy=10):
        a = (x, xs, M, K, ldx, had, w, ws)
        return fl.lib().nvfp4_matvec(*a, g, y, N, ldy, None) if nv else fl.lib().mxfp4_matvec(*a, y, N, ldy, None)

    for kw in (dict(x=None), dict(w=None), dict(ws=None), dict(y=None), dict(M=0), dict(N=0), dict(K=0), dict(ldx=64),
               dict(ldy=9), dict(had=32 if nv else 16), dict(xs=P, had=16 if nv else 32)):
        assert f(**kw) == INVALID, kw
    if nv:
        assert f(g=None) == INVALID and f(g=P + 2) == MISALIGNED
    for kw in (dict(M=17), dict(K=96), dict(ldx=132), dict(xs=P, ldx=136)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=P + 8), dict(w=P + 8), dict(ws=P + 8), dict(y=P + 1), dict(xs=P + 8)):
        assert f(**kw) == MISALIGNED, kw


def test_table_refusals():
    def f(t=P, ld=8, width=8, lens=P, new=P, B=2, free=P, F=8, head=P, page=16, most=8, cu=P, slots=P, nh=P + 64):
        return fl.lib().kv_block_tables(t, ld, width, lens, new, B, free, F, head, page, most, cu, slots, nh, None)

    for kw in (dict(t=None), dict(lens=None), dict(new=None), dict(free=None), dict(head=None), dict(cu=None),
               dict(slots=None), dict(nh=None), dict(B=0), dict(width=0), dict(ld=7), dict(F=0), dict(most=0),
               dict(nh=P)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(page=8), dict(page=48), dict(page=256), dict(B=8193), dict(most=(1 << 30) + 1),
               dict(width=1 << 24, ld=1 << 24, page=128)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(t=P + 2), dict(lens=P + 1), dict(nh=P + 2)):
        assert f(**kw) == MISALIGNED, kw


def test_store_refusals():
    def f(k=P, ldk=256, v=P, ldv=256, s=P, T=4, kc=P, ks=P, vc=P, vs=P, NP=8, H=2, page=16, D=128):
        return fl.lib().kv_fp8_store(k, ldk, v, ldv, s, T, kc, ks, vc, vs, NP, H, page, D, None)

    for kw in (dict(k=None), dict(v=None), dict(s=None), dict(kc=None), dict(ks=None), dict(vc=None), dict(vs=None),
               dict(T=0), dict(H=0), dict(NP=0), dict(D=0), dict(ldk=255), dict(ldv=128)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(D=96, ldk=256, ldv=256), dict(page=24), dict(ldk=260), dict(ldv=260),
               dict(NP=1 << 27), dict(H=32768, ldk=1 << 23, ldv=1 << 23)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(k=P + 8), dict(kc=P + 8), dict(vc=P + 4), dict(s=P + 2)):
        assert f(**kw) == MISALIGNED, kw


def test_attention_refusals():
    def f(q=P, ldq=512, T=4, kc=P, ks=P, vc=P, vs=P, NP=8, page=16, t=P, ldt=8, width=8, lens=P, cu=P, mn=1, ml=100,
          scale=0.1, out=P, B=2, H=2, G=2, D=128, ws=None, wsb=0):
        return fl.lib().kv_fp8_attention(q, ldq, T, kc, ks, vc, vs, NP, page, t, ldt, width, lens, cu, mn, ml, scale,
                                         out, B, H, G, D, ws, wsb, None)

    for kw in (dict(q=None), dict(kc=None), dict(ks=None), dict(vc=None), dict(vs=None), dict(t=None), dict(lens=None),
               dict(cu=None), dict(out=None), dict(B=0), dict(H=0), dict(G=0), dict(T=0), dict(NP=0), dict(width=0),
               dict(ldt=7), dict(mn=0), dict(ml=0), dict(ldq=511), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(ml=129)):  # a table of 8 pages of 16 holds 128 rows
        assert f(**kw) == INVALID, kw
    for kw in (dict(page=20), dict(D=80), dict(G=17, ldq=1 << 13), dict(ldq=516), dict(B=1 << 15, H=4, ldq=1024),
               dict(NP=1 << 27)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(q=P + 8), dict(kc=P + 8), dict(out=P + 8), dict(t=P + 2), dict(ws=P + 8, wsb=1 << 20)):
        assert f(**kw) == MISALIGNED, kw
    L = fl.lib()
    assert L.kv_fp8_attention_workspace_bytes(1, 8, 4, 1, 1000, 96) == 0
    assert L.kv_fp8_attention_workspace_bytes(1, 8, 4, 1, 1000, 128) == 0  # up to 8 splits need none
    assert L.kv_fp8_attention_workspace_bytes(1, 8, 4, 1, 30000, 128) > 0


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_host_tensors_and_non_tensors():
    cache = (z(2, 1, 16, 64, dtype=torch.uint8), z(2, 1, dtype=torch.uint8))
    i = z(4, dtype=torch.int32)
    calls = {
        "x": lambda: fl.rmsnorm_mxfp8(z(4, 64), z(64)),
        "x ": lambda: fl.nvfp4_matvec(z(4, 64), z(8, 32, dtype=torch.uint8), z(512, dtype=torch.uint8), z(1)),
        "block_table": lambda: fl.kv_block_tables(z(4, 4, dtype=torch.int32), i, i, i, i, 16, max_tokens=4),
        "k_new": lambda: fl.kv_fp8_store(z(4, 1, 64), z(4, 1, 64), i, cache, cache),
        "q": lambda: fl.kv_fp8_attention(z(4, 1, 64), cache, cache, z(3, 2, dtype=torch.int32), i, i, max_new=1,
                                         max_len=8),
    }
    for name, call in calls.items():
        with pytest.raises(ValueError, match=f"{name.strip()} must be a CUDA tensor"):
            call()
    with pytest.raises(TypeError, match="x must be a torch.Tensor"):
        fl.rmsnorm_mxfp8(np.zeros((4, 64)), z(64))


def test_reference_block_exponent():
    # the least X with amax <= 448 * 2^X
    assert ref.block_byte([448.0, 448.0001, 224.0, 449 / 2, 0.0, 1e-45, 3e38]).tolist() == [127, 128, 126, 127, 0, 1, 247]


def test_reference_e4m3():
    v = np.array([0.0, -0.0, 448.0, 1e9, -500.0, 2.0 ** -9, 2.0 ** -10, 2.0 ** -10 * 1.01, 17.0, 19.0, np.nan, np.inf])
    want = torch.tensor(np.clip(v, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_bytes(v), want)
    rng = np.random.default_rng(0)
    x = rng.standard_normal(20000).astype(np.float32) * np.exp(rng.standard_normal(20000) * 4).astype(np.float32)
    want = torch.tensor(np.clip(x, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_bytes(x), want)


def test_reference_append_keeps_older_rows_within_half_a_step():
    rng = np.random.default_rng(1)
    codes, byte = np.full((2, 1, 16, 64), 0x7F, np.uint8), np.full((2, 1), 9, np.uint8)
    rows = rng.standard_normal((16, 1, 64)) * 2.0 ** np.arange(16)[:, None, None]
    for t in range(16):
        ref.append(rows[t:t + 1], [16 + t], codes, byte, 16)
    got, top = ref.cache_values(codes[1], byte[1])[0], np.abs(rows).max()
    # one rounding when written (2^-4), and one each time the exponent grew that only subnormals feel
    assert np.all(np.abs(got - rows[:, 0]) <= 2.0 ** -4 * np.abs(rows[:, 0]) + 16 * 2.0 ** -10 * top / 224)
    assert (codes[0] == 0x7F).all() and byte[0] == 9


def test_norms_overlap_check_against_every_byte():
    """summed may be the residual's (x's) own memory or share none of it, which rows of one stride do
    side by side; only where the strides differ does the check go by the whole ranges."""
    from mxfp4_microscaled_bit_b200.serving import _apart
    rng = np.random.default_rng(0)

    def touched(at, ld, rows, cols):
        return {at + 2 * (r * ld + c) + k for r in range(rows) for c in range(cols) for k in (0, 1)}

    seen = set()
    for _ in range(3000):
        rows, cols = int(rng.integers(1, 5)), int(rng.integers(1, 7))
        ld, ld_s = (int(v) for v in cols + rng.integers(0, 9, 2))
        if rng.random() < 0.7:
            ld_s = ld
        lo = 1000
        s = lo + int(rng.integers(-2 * rows * (ld + 1), 2 * rows * (ld + 1)))
        a, b = touched(s, ld_s, rows, cols), touched(lo, ld, rows, cols)
        same = s == lo and (ld_s == ld or rows == 1)
        try:
            _apart("f", s, ld_s, (("x", lo, ld),), rows, cols)
            refused = False
        except ValueError:
            refused = True
        if same or not a & b:
            assert not refused or ld_s != ld and rows > 1, (s, ld_s, ld, rows, cols)
        else:
            assert refused, (s, ld_s, ld, rows, cols)
        seen.add((same, bool(a & b), refused))
    assert seen >= {(True, True, False), (False, True, True), (False, False, False)}
