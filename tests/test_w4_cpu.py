"""4-bit weights without a GPU: the format's reference is pinned, and every call refuses what it
cannot run before it touches the device."""
import ctypes

import numpy as np
import pytest
import torch

import w4_reference as ref
from expert_routed_ffn_softmax_b200 import _abi, build

FAKE = 1 << 20   # an aligned non-null address; never dereferenced
Z, F32 = _abi.MOE_FLAG_W4_ZEROS, _abi.MOE_FLAG_F32_OUT


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def test_quantiser_reference_takes_the_nearest_code():
    """Brute force over the 16 codes: no code's value is nearer than the chosen one's."""
    g = torch.Generator().manual_seed(1)
    w = (torch.randn((2, 128, 16), generator=g) * 0.02).to(torch.bfloat16)
    w[0, :32, 3] = 0          # a group of zeros
    w[1, :, 5] = w[1, :, 5].abs()   # one-sided groups
    for group in (32, 64, 128):
        for zeros in (False, True):
            codes, scales, zp = ref.quantize(w, group, zeros)
            v = ref.values(codes, scales, zp, group)
            idx = torch.arange(128) // group
            s = scales.double()[..., idx].transpose(1, 2)
            z = zp.double()[..., idx].transpose(1, 2)
            every = (torch.arange(16, dtype=torch.float64).view(16, 1, 1, 1) - z) * s
            best = (every - w.double()).abs().amin(0)
            # fp32 division may pick the farther of two codes at a midpoint
            assert bool(((v - w.double()).abs() <= best + 1e-6 * s.abs() + 1e-12).all())
            assert float(v[0, :32, 3].abs().max()) == 0.0


def test_value_formula_by_hand():
    codes = torch.tensor([[[0, 15, 8, 7] + [8] * 60]], dtype=torch.uint8)
    scales = torch.tensor([[[0.5, 2.0]]], dtype=torch.bfloat16)
    v = ref.values(codes, scales, None, 32)[0, :, 0]
    assert v[:4].tolist() == [-4.0, 3.5, 0.0, -0.5] and float(v[32]) == 0.0
    zp = torch.tensor([[[3, 10]]], dtype=torch.uint8)
    v = ref.values(codes, scales, zp, 32)[0, :, 0]
    assert v[:4].tolist() == [-1.5, 6.0, 2.5, 2.0] and float(v[32]) == -4.0


def test_packed_bytes(lib):
    n = lib.moe_w4_packed_bytes
    assert n(1, 64, 16, 64, 0) == 544
    assert n(1, 64, 16, 32, 0) == 576
    assert n(1, 64, 16, 128, Z) == 560
    assert n(1, 64, 16, 32, Z) == 608
    assert n(128, 2816, 704, 64, 0) == 128 * 44 * 44 * 544
    assert n(1, 16384, 1048576, 64, 0) == 256 * 65536 * 544     # past 32 bits
    for bad in ((1, 96, 16, 64, 0), (1, 64, 24, 64, 0), (1, 64, 16, 48, 0), (0, 64, 16, 64, 0),
                (1, 32768, 16, 64, 0), (1, 64, 2097152, 64, 0), (8192, 64, 16, 64, 0),
                (1, 64, 16, 64, F32), (1, 0, 16, 64, 0), (1, 64, 0, 64, 0)):
        assert n(*bad) == 0, bad


def test_weight_calls_refuse(lib):
    INV, UNS = _abi.MOE_ERR_INVALID_ARG, _abi.MOE_ERR_UNSUPPORTED
    p = lib.moe_w4_pack
    assert p(FAKE, FAKE, None, 0, 64, 16, 64, FAKE, None) == 0
    assert p(None, FAKE, None, 1, 64, 16, 64, FAKE, None) == INV
    assert p(FAKE, None, None, 1, 64, 16, 64, FAKE, None) == INV
    assert p(FAKE, FAKE, None, 1, 64, 16, 64, None, None) == INV
    assert p(FAKE + 8, FAKE, None, 1, 64, 16, 64, FAKE, None) == INV     # misaligned codes
    assert p(FAKE, FAKE + 1, None, 1, 64, 16, 64, FAKE, None) == INV
    assert p(FAKE, FAKE, None, 1, 64, 16, 48, FAKE, None) == INV          # group
    assert p(FAKE, FAKE, None, 1, 96, 16, 64, FAKE, None) == UNS
    assert p(FAKE, FAKE, None, -1, 64, 16, 64, FAKE, None) == INV
    for f in (lib.moe_w4_quantize_weights, lib.moe_w4_dequantize_weights):
        assert f(FAKE, 0, 64, 16, 64, 0, FAKE, None) == 0
        assert f(None, 1, 64, 16, 64, 0, FAKE, None) == INV
        assert f(FAKE, 1, 64, 16, 64, 0, None, None) == INV
        assert f(FAKE, 1, 64, 16, 64, 1, FAKE, None) == INV               # flag
        assert f(FAKE, 1, 64, 16, 16, 0, FAKE, None) == INV
        assert f(FAKE + 2, 1, 64, 16, 64, 0, FAKE, None) == INV
        assert f(FAKE, 1, 64, 20, 64, Z, FAKE, None) == UNS


def test_linear_refuses(lib):
    f = lib.moe_linear_w4
    ws = lib.moe_linear_w4_workspace_size
    assert ws(1, 2816) == 0 and ws(8, 128) == 0                # kept in shared memory
    assert ws(16, 2816) >= 2 * 16 * 2816 and ws(8, 16384) >= 2 * 8 * 16384
    assert ws(0, 128) == 0 and ws(17, 128) == 0 and ws(8, 100) == 0
    ok = dict(x=FAKE, w=FAKE, T=8, K=128, N=64, group=64, flags=0, y=FAKE + 4096, ws=None, n=0)

    def rc(**kw):
        a = {**ok, **kw}
        return f(a["x"], a["w"], a["T"], a["K"], a["N"], a["group"], a["flags"], a["y"], a["ws"],
                 a["n"], None)
    assert rc(T=0) == 0
    assert rc(T=16, K=4096) == _abi.MOE_ERR_INVALID_ARG         # needs a workspace
    assert rc(T=16, K=4096, ws=FAKE + 8, n=1 << 30) == _abi.MOE_ERR_INVALID_ARG
    assert rc(T=16, K=4096, ws=FAKE, n=1024) == _abi.MOE_ERR_NO_WORKSPACE
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(x=FAKE + 2), dict(w=FAKE + 8),
               dict(y=FAKE + 4), dict(y=FAKE), dict(T=-1), dict(group=16), dict(flags=1),
               dict(K=0), dict(N=-16)):
        assert rc(**kw) == _abi.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(T=17), dict(K=100), dict(K=16448), dict(N=72), dict(N=1048592)):
        assert rc(**kw) == _abi.MOE_ERR_UNSUPPORTED, kw


def test_dense_refuses(lib):
    f, ws = lib.moe_dense_ffn_w4, lib.moe_dense_w4_workspace_size
    assert ws(8, 2816, 2112) >= 2 * 8 * 2112
    for bad in ((0, 2816, 2112), (17, 2816, 2112), (8, 2800, 2112), (8, 2816, 2100),
                (8, 32768, 2112), (8, 2816, 16384)):
        assert ws(*bad) == 0, bad
    ok = dict(x=FAKE, g=FAKE, u=FAKE, d=FAKE, T=8, H=2816, I=2112, group=64, flags=0,
              y=FAKE + 4096, ws=FAKE, n=1 << 30)

    def rc(**kw):
        a = {**ok, **kw}
        return f(a["x"], a["g"], a["u"], a["d"], a["T"], a["H"], a["I"], a["group"], a["flags"],
                 a["y"], a["ws"], a["n"], None)
    assert rc(T=0) == 0
    for kw in (dict(x=None), dict(g=None), dict(u=None), dict(d=None), dict(y=None), dict(ws=None),
               dict(u=FAKE + 4), dict(y=FAKE), dict(group=0), dict(flags=F32), dict(T=-1)):
        assert rc(**kw) == _abi.MOE_ERR_INVALID_ARG, kw
    assert rc(T=17) == _abi.MOE_ERR_UNSUPPORTED
    assert rc(I=2100) == _abi.MOE_ERR_UNSUPPORTED
    assert rc(n=256) == _abi.MOE_ERR_NO_WORKSPACE


def test_layer_refuses(lib):
    f, ws = lib.moe_forward_w4, lib.moe_w4_workspace_size
    assert ws(8, 2816, 128, 704, 8, 0) >= 64 * (2 * 704 + 4 * 2816)
    for bad in ((17, 2816, 128, 704, 8, 0), (8, 2816, 128, 700, 8, 0), (8, 2816, 260, 704, 8, 0),
                (8, 2816, 128, 704, 9, 0), (8, 2816, 128, 704, 8, _abi.MOE_FLAG_FFN_PAIRS),
                (0, 2816, 128, 704, 8, 0)):
        assert ws(*bad) == 0, bad
    ok = dict(x=FAKE, r=FAKE, g=FAKE, u=FAKE, d=FAKE, T=8, H=2816, E=128, I=704, k=8, group=64,
              flags=0, y=FAKE + 4096, ws=FAKE, n=1 << 30)

    def rc(**kw):
        a = {**ok, **kw}
        return f(a["x"], a["r"], None, a["g"], a["u"], a["d"], a["T"], a["H"], a["E"], a["I"],
                 a["k"], a["group"], a["flags"], a["y"], None, a["ws"], a["n"], None)
    assert rc(T=0) == 0
    for kw in (dict(x=None), dict(r=None), dict(g=None), dict(d=None), dict(y=FAKE), dict(ws=None),
               dict(k=0), dict(k=9, E=8), dict(group=96), dict(flags=F32),
               dict(flags=_abi.MOE_FLAG_ROUTER_SCREEN), dict(d=FAKE + 8), dict(T=-3)):
        assert rc(**kw) == _abi.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(T=17), dict(I=700), dict(E=6, k=2), dict(k=9)):
        assert rc(**kw) == _abi.MOE_ERR_UNSUPPORTED, kw
    assert rc(n=1024) == _abi.MOE_ERR_NO_WORKSPACE


def test_binding_refuses_without_a_device(lib):
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    for call in (lambda: _abi.linear_w4(x, None), lambda: _abi.w4_quantize(x),
                 lambda: _abi.dense_ffn_w4(x, None, None, None), lambda: _abi.w4_dequantize(None),
                 lambda: _abi.forward_w4(x, x, None, None, None, 1)):
        with pytest.raises(TypeError, match="CUDA"):
            call()


def test_reciprocal_products_round_like_quotients():
    """The quantiser multiplies by the reciprocal, in one fused operation that also rounds to a
    multiple of 2^-11, and then rounds to an integer: for every pair of 8-bit significands and every
    exponent that gives a quotient up to 16 that is the rounded quotient, ties included."""
    f32 = np.float32
    snap, rnd = 1.5 * 2.0 ** 12, 1.5 * 2.0 ** 23
    a = np.arange(128, 256, dtype=np.float64)[:, None]
    for b in range(128, 256):
        inv = f32(1) / f32(b)
        for e in range(-8, 5):
            x = a * 2.0 ** e
            x = x[x / b <= 16]
            # the product has 32 bits and the sum ends above 2^-29 of it: exact in float64 until it is
            # rounded to fp32, as the fused operation does
            snapped = (x * np.float64(inv) + snap).astype(f32)
            got = (snapped.astype(np.float64) + (rnd - snap)).astype(f32).astype(np.float64) - rnd
            assert np.array_equal(got, np.rint(x / b))


def test_packed_reference_round_trip():
    """Every code, scale and zero point of the reference packing is where the header says."""
    codes, scales, zp = ref.make_checkpoint(1, 128, 32, 32, True, seed=3)
    p = ref.packed_bytes(codes, scales, zp, 32)
    assert p.shape == (1, 2, 2, 608)
    sc = scales.view(torch.int16).numpy().view(np.uint16)
    for n, k in ((0, 0), (8, 1), (31, 127), (17, 70), (15, 63), (16, 32)):
        rec = p[0, n // 16, k // 64]
        r, kk = n % 16, k % 64
        t, j = (kk % 32) // 8, kk % 8
        word = rec[16 * (4 * (r % 8) + t) + 8 * (kk // 32) + 4 * (r // 8):][:4].view("<u4")[0]
        nib = (int(word) >> (4 * ((j >> 1) + 4 * (j & 1)))) & 15
        assert nib == int(codes[0, n, k])
        slot, q = 2 * (r % 8) + r // 8, kk // 32
        assert rec[512 + 32 * q + 2 * slot:][:2].view("<u2")[0] == sc[0, n, k // 32]
        assert rec[512 + 64 + 16 * q + slot] == int(zp[0, n, k // 32])
