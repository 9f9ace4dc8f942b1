"""The 4-bit weight format and the operators on it, written from their definitions in float64
(numpy / torch on the CPU), with bounds on what an implementation in fp32 may be off by.

Shared by test_w4_cpu.py and test_w4_gpu.py; it uses nothing of the library."""
import math

import numpy as np
import torch

U32 = 2.0 ** -23     # one fp32 addition inside a tensor-core product may truncate: a whole step
HALF_BF16 = 2.0 ** -8


def groups(K, group):
    return -(-K // group)


def make_checkpoint(E, K, N, group, zeros, seed, extreme=False):
    """codes uint8 [E, N, K] (one per element), scales bf16 [E, N, G], zeros uint8 [E, N, G]."""
    g = torch.Generator().manual_seed(seed)
    G = groups(K, group)
    if extreme:   # only the ends of the code range
        codes = torch.randint(0, 2, (E, N, K), generator=g) * 15
        zp = torch.randint(0, 2, (E, N, G), generator=g) * 15
    else:
        codes = torch.randint(0, 16, (E, N, K), generator=g)
        zp = torch.randint(0, 16, (E, N, G), generator=g)
    scales = (torch.rand((E, N, G), generator=g) + 0.25) * 0.01
    scales *= torch.where(torch.rand((E, N, G), generator=g) < 0.2, -1.0, 1.0)   # any finite scale
    return (codes.to(torch.uint8), scales.to(torch.bfloat16),
            zp.to(torch.uint8) if zeros else None)


def nibbles(codes):
    """One code per byte [..., K] -> packed bytes [..., K/2], element 2b in the low nibble."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def values(codes, scales, zeros, group):
    """float64 [E, K, N]: (code - zero) * scale."""
    K = codes.shape[-1]
    idx = torch.arange(K) // group
    z = 8.0 if zeros is None else zeros.to(torch.float64)[..., idx]
    return ((codes.to(torch.float64) - z) * scales.to(torch.float64)[..., idx]).transpose(1, 2)


def packed_bytes(codes, scales, zeros, group):
    """The records of include/moe.h: uint8 numpy [E, N/16, K/64, R]."""
    c = codes.numpy()
    E, N, K = c.shape
    g = 2 if group == 32 else 1
    R = 512 + g * (48 if zeros is not None else 32)
    out = np.zeros((E, N // 16, K // 64, R), np.uint8)
    order = [0, 2, 4, 6, 1, 3, 5, 7]
    rows = [r for i in range(8) for r in (i, i + 8)]
    sc = scales.view(torch.int16).numpy().view(np.uint16)
    for s in range(N // 16):
        for b in range(K // 64):
            blk = c[:, 16 * s:16 * s + 16, 64 * b:64 * b + 64].astype(np.uint32)
            rec = out[:, s, b]
            for i in range(8):
                for t in range(4):
                    for w, (r, k) in enumerate(((i, 0), (i + 8, 0), (i, 32), (i + 8, 32))):
                        e = blk[:, r, k + 8 * t:k + 8 * t + 8]
                        word = sum(e[:, order[p]] << (4 * p) for p in range(8)).astype("<u4")
                        at = 16 * (4 * i + t) + 4 * w
                        rec[:, at:at + 4] = word.view(np.uint8).reshape(E, 4)
            for q in range(g):
                gi = (64 * b + 32 * q) // group
                v = np.ascontiguousarray(sc[:, 16 * s:16 * s + 16, gi][:, rows].astype("<u2"))
                rec[:, 512 + 32 * q:544 + 32 * q] = v.view(np.uint8).reshape(E, 32)
                if zeros is not None:
                    z = zeros.numpy()[:, 16 * s:16 * s + 16, gi][:, rows]
                    rec[:, 512 + 32 * g + 16 * q:528 + 32 * g + 16 * q] = z
    return out


def quantize(w, group, zeros):
    """bf16 w [E, K, N] -> codes [E, N, K], scales bf16 [E, N, G], zero points [E, N, G], by the
    documented fp32 steps (IEEE single precision through numpy)."""
    v = w.float().numpy().transpose(0, 2, 1)
    E, N, K = v.shape
    G = groups(K, group)
    codes = np.empty((E, N, K), np.uint8)
    scales = torch.empty((E, N, G), dtype=torch.bfloat16)
    zp = np.full((E, N, G), 8, np.uint8)
    for g in range(G):
        p = v[:, :, g * group:(g + 1) * group]
        lo, hi = np.minimum(p.min(2), np.float32(0)), np.maximum(p.max(2), np.float32(0))
        s = (hi - lo) / np.float32(15) if zeros else np.maximum(-lo, hi) / np.float32(7)
        sb = torch.from_numpy(s).to(torch.bfloat16)
        scales[:, :, g] = sb
        s = sb.float().numpy()
        with np.errstate(divide="ignore", invalid="ignore"):
            z = np.where(s > 0, np.clip(np.rint(-lo / s), 0, 15) if zeros else 8.0, 8.0)
            q = np.where(s[..., None] > 0, np.rint(p / s[..., None]) + z[..., None], 8.0)
        zp[:, :, g] = z
        codes[:, :, g * group:(g + 1) * group] = np.clip(q, 0, 15)
    return torch.from_numpy(codes), scales, torch.from_numpy(zp)


# ----------------------------------------------------------------------------- operators
def sum_steps(K, group):
    """fp32 roundings on the way of one output: the products' sums (at most one per 8 elements),
    two per group (scale, add), and the joins of partial sums."""
    return K / 8 + 2 * groups(K, min(group, 64)) + 32


def linear(x, v, group):
    """float64 y and a bound on an fp32 implementation's error before the output's rounding."""
    x = x.to(torch.float64)
    return x @ v, sum_steps(v.shape[0], group) * U32 * (x.abs() @ v.abs())


def gelu_tanh(a):
    return 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a ** 3)))


def ffn(x, wg, wu, wd, group):
    """GEGLU FFN in float64 and a bound on an implementation's error before the output's
    rounding: fp32 sums; tanh good to 2^-10.9 (the hardware's approximation) and a few fp32
    steps; h rounded to bf16; fp32 sums again.  |gelu'| <= 1.13."""
    (g, eg), (u, eu) = linear(x, wg, group), linear(x, wu, group)
    a = gelu_tanh(g)
    h = a * u
    ea = 1.13 * eg + 0.5 * g.abs() * 2.0 ** -10.9 + 8 * U32 * a.abs()
    eh = ea * (u.abs() + eu) + a.abs() * eu + 2 * U32 * h.abs()
    eh = eh + HALF_BF16 * (h.abs() + eh)
    y, ey = h @ wd, sum_steps(wd.shape[0], group) * U32 * ((h.abs() + eh) @ wd.abs())
    return y, ey + eh @ wd.abs()


def rounded(y, err, dtype):
    """The bound after the output's own rounding."""
    half = {torch.bfloat16: HALF_BF16, torch.float32: 2.0 ** -24}[dtype]
    return err + half * (y.abs() + err) + 1e-38


def layer(x, ids, weights, wg, wu, wd, group):
    """The routed layer in float64 for given ids [T, k] and weights [T, k], and a bound as above;
    weights may be off by 1e-5 (the router's tolerance)."""
    T, k = ids.shape
    y = torch.zeros((T, wd.shape[2]), dtype=torch.float64)
    err = torch.zeros_like(y)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            o, eo = ffn(x[t:t + 1], wg[e], wu[e], wd[e], group)
            w = float(weights[t, j])
            y[t] += w * o[0]
            err[t] += w * eo[0] + 1e-5 * (o[0].abs() + eo[0]) + (k + 1) * U32 * w * o[0].abs()
    return y, err


def check(got, y, err, what=""):
    """Every element of `got` lies within the bound of the float64 value."""
    bound = rounded(y, err, got.dtype)
    diff = (got.cpu().to(torch.float64) - y).abs()
    bad = ~(diff <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((diff / bound).nan_to_num(1e9).max()))
