"""The 4-bit weight-only (W4A16) operators for batches of a few tokens, as cases to time and check.

Weights are 4-bit codes with one bf16 scale (and, in the asymmetric form, one zero point) per
group of `group` consecutive elements along the reduction axis; activations stay bf16:

    linear   y = x W
    dense    y = (gelu_tanh(x Wg) * (x Wu)) Wd            the dense MLP beside the MoE
    moe      the whole routed layer: softmax top-k router, GEGLU experts, weighted sum
    weights  bf16 weights to 4 bits and back (the bf16 copy that large batches run on)

`own` chooses between the framework's calls and the plain form (elementary torch operations in
32 bits; the router's logits in 64, since a ranking is decided on them).
"""
import math

import numpy as np
import torch

own = False

WEIGHT_STD = 0.02


def listed():
    return [
        # one expert's down projection for one token: the smallest call, where latency counts
        dict(name="linear_t1_small", op="linear", T=1, K=704, N=2816, group=32, zeros=False,
             fp32=False),
        # the dense MLP's down projection for an odd batch, asymmetric codes
        dict(name="linear_t7_dense_down", op="linear", T=7, K=2112, N=2816, group=64, zeros=True,
             fp32=False),
        # a square projection of a wide model for the largest batch
        dict(name="linear_t16_wide", op="linear", T=16, K=8192, N=8192, group=128, zeros=False,
             fp32=False),
        # a vocabulary projection for one token, logits in fp32
        dict(name="linear_t1_vocab", op="linear", T=1, K=2816, N=262144, group=128, zeros=False,
             fp32=True),
        # the dense MLP of one layer for one token
        dict(name="dense_t1", op="dense", T=1, H=2816, I=2112, group=64, zeros=False),
        # the same for the decode batch, small groups and zero points
        dict(name="dense_t8_zeros", op="dense", T=8, H=2816, I=2112, group=32, zeros=True),
        # a wide dense MLP for an odd batch
        dict(name="dense_t13_wide", op="dense", T=13, H=4096, I=8192, group=128, zeros=False),
        # the routed layer for one token
        dict(name="moe_t1", op="moe", T=1, H=2816, I=704, E=128, k=8, group=64, zeros=False,
             bias=False, renorm=True),
        # the decode batch
        dict(name="moe_t8", op="moe", T=8, H=2816, I=704, E=128, k=8, group=64, zeros=False,
             bias=False, renorm=True),
        # the largest batch, skewed routing, zero points, raw softmax weights
        dict(name="moe_t16_skewed", op="moe", T=16, H=2816, I=704, E=128, k=8, group=32,
             zeros=True, bias=True, renorm=False),
        # the weights of one dense projection
        dict(name="weights_dense", op="weights", E=1, K=2816, N=2112, group=64, zeros=True),
        # one projection of all experts of a layer
        dict(name="weights_experts", op="weights", E=128, K=2816, N=704, group=32, zeros=False),
    ]


def _spread(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("linear", "dense", "moe", "weights"))
    case = dict(op=op, group=rng.choice((32, 64, 128)), zeros=rng.random() < 0.5)
    if op == "linear":
        K = _spread(rng, 64, 16384, 64)
        N = _spread(rng, 16, min(262144, 2816 * 262144 // K // 16 * 16), 16)
        case.update(T=rng.randint(1, 16), K=K, N=N, fp32=rng.random() < 0.5)
    elif op == "dense":
        H = _spread(rng, 64, 8192, 64)
        case.update(T=rng.randint(1, 16), H=H, I=_spread(rng, 64, 8192, 64))
    elif op == "moe":
        E = rng.choice((4 * rng.randint(1, 32), 8 * rng.randint(17, 32)))
        H = _spread(rng, 64, 4096, 64)
        most = 128 * 2816 * 704 // (E * H)
        case.update(T=rng.randint(1, 16), H=H, I=_spread(rng, 64, max(64, min(2048, most // 64 * 64)), 64),
                    E=E, k=rng.randint(1, min(8, E)), bias=rng.random() < 0.5,
                    renorm=rng.random() < 0.7)
    else:
        K = _spread(rng, 64, 8192, 64)
        N = _spread(rng, 16, 8192, 16)
        E = rng.randint(1, max(1, min(64, 128 * 2816 * 704 // (K * N))))
        case.update(E=E, K=K, N=N)
    return case


# ----------------------------------------------------------------------------- inputs
def _bf16_weights(g, E, K, N):
    """bf16 weights [E, K, N] as a trained layer has them: about normal, a small spread."""
    w = torch.randn((E, K, N), generator=g, device="cuda", dtype=torch.float32)
    return w.mul_(WEIGHT_STD).to(torch.bfloat16)


def _checkpoint(g, E, K, N, group, zeros):
    """A 4-bit matrix as a checkpoint holds it: codes uint8 [E, N, K/2] (element 2b in the low
    nibble), scales bf16 [E, N, G], zero points uint8 [E, N, G] or None.  The codes are those
    of normal weights scaled by their group's range."""
    G = -(-K // group)
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, N, G), dtype=torch.bfloat16, device="cuda")
    zp = torch.empty((E, N, G), dtype=torch.uint8, device="cuda") if zeros else None
    step = max(1, (1 << 27) // (N * K)) if E > 1 else 1
    for e in range(0, E, step):
        n = min(step, E - e)
        w = torch.randn((n, N, K), generator=g, device="cuda", dtype=torch.float32)
        spread = torch.rand((n, N, G), generator=g, device="cuda") + 0.5
        q = (w * 2.5).round_()
        if zeros:
            z = torch.randint(5, 11, (n, N, G), generator=g, device="cuda")
            zp[e:e + n] = z.to(torch.uint8)
            q += z.repeat_interleave(group, 2)[:, :, :K]
        else:
            q += 8
        q = q.clamp_(0, 15).to(torch.uint8).view(n, N, K // 2, 2)
        codes[e:e + n] = q[..., 0] | (q[..., 1] << 4)
        scales[e:e + n] = (spread * (WEIGHT_STD / 2.5)).to(torch.bfloat16)
        del w, spread, q
    return dict(codes=codes, scales=scales, zeros=zp, K=K, group=group)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], dict(case=case)
    if op == "weights":
        s["w"] = _bf16_weights(g, case["E"], case["K"], case["N"])
        return s
    width = case["K"] if op == "linear" else case["H"]
    s["x"] = torch.randn((case["T"], width), generator=g, device="cuda").to(torch.bfloat16)
    form = (case["group"], case["zeros"])
    if op == "linear":
        s["mats"] = dict(w=_checkpoint(g, 1, case["K"], case["N"], *form))
        return s
    E = case["E"] if op == "moe" else 1
    s["mats"] = dict(gate=_checkpoint(g, E, case["H"], case["I"], *form),
                     up=_checkpoint(g, E, case["H"], case["I"], *form),
                     down=_checkpoint(g, E, case["I"], case["H"], *form))
    if op == "moe":
        s["router"] = _bf16_weights(g, 1, case["H"], E)[0]
        s["bias"] = torch.from_numpy(_bias(E)).cuda() if case["bias"] else None
    return s


def _bias(E):
    """A router bias that skews the load: 2 ln(1 / (e + 1))."""
    return (-2.0 * np.log(np.arange(1, E + 1, dtype=np.float64))).astype(np.float32)


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and "mats" in s:
        # the weights in the library's layout, laid out once when a checkpoint is loaded
        import expert_routed_ffn_softmax_b200 as moe
        s["packed"] = {n: moe.w4_pack(m["codes"], m["scales"], m["zeros"], group=m["group"])
                       for n, m in s["mats"].items()}
    return s


# ----------------------------------------------------------------------------- the framework's calls
def _run_own(s):
    import expert_routed_ffn_softmax_b200 as moe
    case = s["case"]
    op = case["op"]
    if op == "weights":
        return moe.w4_dequantize(moe.w4_quantize(s["w"], group=case["group"], zeros=case["zeros"]))
    p = s["packed"]
    if op == "linear":
        return moe.linear_w4(s["x"], p["w"], fp32=case["fp32"])
    if op == "dense":
        return moe.dense_ffn_w4(s["x"], p["gate"], p["up"], p["down"])
    return moe.forward_w4(s["x"], s["router"], p["gate"], p["up"], p["down"], case["k"],
                          bias=s["bias"], renorm=case["renorm"])


# ----------------------------------------------------------------------------- the plain form
def _values(m, rows=None):
    """The weights that a checkpoint's codes stand for, fp32 [E (or rows), N, K]."""
    codes, scales, zeros = m["codes"], m["scales"], m["zeros"]
    if rows is not None:
        codes, scales = codes[rows], scales[rows]
        zeros = None if zeros is None else zeros[rows]
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.float32)
    wide = lambda t: t.to(torch.float32).repeat_interleave(m["group"], -1)[..., :m["K"]]  # noqa: E731
    return (q - (8.0 if zeros is None else wide(zeros))) * wide(scales)


def _gelu_tanh(a):
    return 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a * a * a)))


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "weights":
        return _weights_plain(s["w"], case["group"], case["zeros"])
    x, m = s["x"].to(torch.float32), s["mats"]
    if op == "linear":
        y = x @ _values(m["w"])[0].t()
        return y if case["fp32"] else y.to(torch.bfloat16)
    if op == "dense":
        h = _gelu_tanh(x @ _values(m["gate"])[0].t()) * (x @ _values(m["up"])[0].t())
        return (h @ _values(m["down"])[0].t()).to(torch.bfloat16)
    # the router: its ranking is decided in 64 bits
    logits = s["x"].to(torch.float64) @ s["router"].to(torch.float64)
    if s["bias"] is not None:
        logits = logits + s["bias"].to(torch.float64)
    ids = torch.sort(-logits, dim=1, stable=True).indices[:, :case["k"]]
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    picked = torch.gather(e, 1, ids)
    w = picked / (picked if case["renorm"] else e).sum(1, keepdim=True)
    # every (token, slot) pair with its expert's weights
    pairs = ids.flatten()
    xp = x.repeat_interleave(case["k"], 0).unsqueeze(-1)
    h = (_gelu_tanh(torch.bmm(_values(m["gate"], pairs), xp))
         * torch.bmm(_values(m["up"], pairs), xp))
    o = torch.bmm(_values(m["down"], pairs), h).view(case["T"], case["k"], -1)
    return (o * w.to(torch.float32).unsqueeze(-1)).sum(1).to(torch.bfloat16)


def _weights_plain(w, group, zeros):
    E, K, N = w.shape
    G = -(-K // group)
    v = w.to(torch.float32)
    pad = v.new_zeros((E, G * group - K, N))
    v = torch.cat((v, pad), 1).view(E, G, group, N)
    if zeros:
        lo, hi = v.amin(2).clamp(max=0), v.amax(2).clamp(min=0)
        s = ((hi - lo) / 15.0).to(torch.bfloat16).to(torch.float32)
        z = torch.where(s > 0, (-lo / s).round().clamp(0, 15), torch.full_like(s, 8.0))
    else:
        s = (v.abs().amax(2) / 7.0).to(torch.bfloat16).to(torch.float32)
        z = torch.full_like(s, 8.0)
    s, z = s.unsqueeze(2), z.unsqueeze(2)
    q = torch.where(s > 0, (v / s).round() + z, z).clamp(0, 15)
    return ((q - z) * s).view(E, G * group, N)[:, :K].to(torch.bfloat16)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------- the work
def _mat_bytes(case, K, N):
    G = -(-K // case["group"])
    return K * N / 2 + N * G * (3 if case["zeros"] else 2)


def _active(case):
    """Experts that a batch reaches on average (routing of normal activations)."""
    rng = np.random.default_rng(0)
    L = rng.standard_normal((16, case["T"], case["E"])) * (WEIGHT_STD * math.sqrt(case["H"]))
    if case["bias"]:
        L = L + _bias(case["E"])
    top = np.argsort(-L, axis=2)[:, :, :case["k"]]
    return float(np.mean([len(np.unique(t)) for t in top]))


def work(case):
    op = case["op"]
    if op == "weights":
        n = case["E"] * case["K"] * case["N"]
        # bf16 in, 4 bits out; 4 bits in, bf16 out
        return dict(bytes=4.0 * n + 2 * case["E"] * _mat_bytes(case, case["K"], case["N"]),
                    flops=4.0 * n)
    T = case["T"]
    if op == "linear":
        K, N = case["K"], case["N"]
        return dict(bytes=_mat_bytes(case, K, N) + 2.0 * T * K + (4.0 if case["fp32"] else 2.0) * T * N,
                    flops=2.0 * T * K * N)
    H, I = case["H"], case["I"]
    mats = 2 * _mat_bytes(case, H, I) + _mat_bytes(case, I, H)
    if op == "dense":
        return dict(bytes=mats + 4.0 * T * H, flops=6.0 * T * H * I)
    E, k = case["E"], case["k"]
    return dict(bytes=_active(case) * mats + 2.0 * H * E + 4.0 * T * H,
                flops=6.0 * T * k * H * I + 2.0 * T * H * E)


# ----------------------------------------------------------------------------- 64 bits
def _matrix64(m, e):
    """One checkpoint matrix as float64 [K, N], nibble by nibble from the format's definition."""
    c = m["codes"][e]
    N, K, group = c.shape[0], m["K"], m["group"]
    out = torch.empty((K, N), dtype=torch.float64, device=c.device)
    out[0::2] = (c % 16).t().to(torch.float64)
    out[1::2] = (c // 16).t().to(torch.float64)
    for i in range(m["scales"].shape[2]):
        part = out[i * group:(i + 1) * group]
        part -= 8.0 if m["zeros"] is None else m["zeros"][e, :, i].to(torch.float64)
        part *= m["scales"][e, :, i].to(torch.float64)
    return out


def _gelu64(a):
    return a / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (a + 0.044715 * a ** 3)))


def _ffn64(x, m, e):
    g, u = x @ _matrix64(m["gate"], e), x @ _matrix64(m["up"], e)
    return (_gelu64(g) * u) @ _matrix64(m["down"], e)


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "weights":
        return _weights64(s["w"], case["group"], case["zeros"])
    x, m = s["x"].to(torch.float64), s["mats"]
    if op == "linear":
        return x @ _matrix64(m["w"], 0)
    if op == "dense":
        return _ffn64(x, m, 0)
    logits = (x @ s["router"].to(torch.float64)).cpu().numpy()
    if s["bias"] is not None:
        logits = logits + s["bias"].to(torch.float64).cpu().numpy()
    y = torch.zeros_like(x)
    of = {}
    for t in range(case["T"]):
        order = sorted(range(case["E"]), key=lambda e: (-logits[t, e], e))[:case["k"]]
        p = np.exp(logits[t] - logits[t].max())
        p /= p[order].sum() if case["renorm"] else p.sum()
        for e in order:
            of.setdefault(e, []).append((t, float(p[e])))
    for e, pairs in of.items():
        rows = torch.tensor([t for t, _ in pairs], device=x.device)
        w = torch.tensor([v for _, v in pairs], device=x.device, dtype=torch.float64)
        y.index_add_(0, rows, w[:, None] * _ffn64(x[rows], m, e))
    return y


def _weights64(w, group, zeros):
    """Scale and zero point of each group, every weight to the nearest code's value."""
    out = torch.empty(w.shape, dtype=torch.float64, device=w.device)
    for k0 in range(0, w.shape[1], group):
        v = w[:, k0:k0 + group].to(torch.float64)
        if zeros:
            lo = torch.minimum(v.min(1, keepdim=True).values, v.new_zeros(1))
            hi = torch.maximum(v.max(1, keepdim=True).values, v.new_zeros(1))
            step = ((hi - lo) / 15).to(torch.bfloat16).to(torch.float64)
            zero = torch.nan_to_num(torch.round(-lo / step), nan=8.0).clamp(0, 15)
        else:
            step = (v.abs().max(1, keepdim=True).values / 7).to(torch.bfloat16).to(torch.float64)
            zero = torch.full_like(step, 8.0)
        level = torch.nan_to_num(torch.round(v / step), nan=0.0)
        out[:, k0:k0 + group] = (torch.minimum(torch.maximum(level, -zero), 15 - zero)) * step
    return out
