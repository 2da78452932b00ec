"""What is measured of the operators around the quantized linear layer of a
diffusion network: group norm with an activation on channels-last maps (forward,
gradients, and as the producer of the layer's int8 codes), and the low-rank
adapters of many requests beside the layer (forward and gradients).

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is true, through this repository's public entry points.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # group norm + SiLU in front of a layer of the lowest-resolution stage
        # (8 x 8 maps, one classifier-free-guidance pair): latency
        {"name": "norm_8x8_pair", "op": "norm", "B": 2, "S": 64, "C": 1280, "G": 32, "act": "silu", "dtype": "bf16"},
        # fp32 maps of odd size without an activation (norm in front of an attention projection)
        {"name": "norm_33x31_fp32", "op": "norm", "B": 3, "S": 1023, "C": 1152, "G": 32, "act": "none", "dtype": "fp32"},
        # full-resolution maps of an image decoder: far more than fits on chip
        {"name": "norm_256x256", "op": "norm", "B": 2, "S": 65536, "C": 256, "G": 32, "act": "silu", "dtype": "bf16"},
        # gradients at an inner stage, and on large odd maps
        {"name": "norm_bwd_32x32", "op": "norm_bwd", "B": 8, "S": 1024, "C": 640, "G": 32, "act": "silu", "dtype": "bf16"},
        {"name": "norm_bwd_127x127", "op": "norm_bwd", "B": 3, "S": 16129, "C": 320, "G": 32, "act": "silu", "dtype": "bf16"},
        # norm -> codes -> quantized linear -> adapters, one request per image
        {"name": "block_16x16", "op": "block", "B": 4, "S": 256, "C": 1152, "G": 32, "act": "none", "N": 1152, "L": 2, "R": 16, "Q": 4},
        {"name": "block_32x32", "op": "block", "B": 8, "S": 1024, "C": 2304, "G": 32, "act": "silu", "N": 3456, "L": 4, "R": 32, "Q": 8},
        # one conditioning vector per request (modulation layers): latency
        {"name": "adapter_64_rows", "op": "adapter", "M": 64, "K": 1152, "N": 3456, "L": 16, "R": 16, "Q": 64, "ragged": False, "dtype": "bf16"},
        # the MLP down projection of 32 images of 256 tokens with 8 adapters
        {"name": "adapter_fc2", "op": "adapter", "M": 8192, "K": 4608, "N": 1152, "L": 8, "R": 64, "Q": 32, "ragged": False, "dtype": "bf16"},
        # requests of very different lengths, some without an adapter
        {"name": "adapter_ragged_qkv", "op": "adapter", "M": 16384, "K": 2304, "N": 3456, "L": 6, "R": 32, "Q": 23, "ragged": True, "dtype": "bf16"},
        # training of the adapters beside the frozen layer
        {"name": "adapter_bwd_fc2", "op": "adapter_bwd", "M": 8192, "K": 4608, "N": 1152, "L": 4, "R": 16, "Q": 32, "ragged": False, "dtype": "bf16"},
        {"name": "adapter_bwd_ragged_fp32", "op": "adapter_bwd", "M": 777, "K": 1152, "N": 2304, "L": 3, "R": 8, "Q": 9, "ragged": True, "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["norm", "norm", "norm_bwd", "block", "adapter", "adapter", "adapter_bwd"])
    if op in ("norm", "norm_bwd"):
        G = rng.choice([8, 16, 32])
        C = G * rng.choice([4, 8, 10, 20, 30, 36, 40])
        B = _log(rng, 1, 16)
        top = (1 << 25) if op == "norm" else (1 << 24)
        S = _log(rng, 16, max(17, min(66000, top // (B * C))))
        return {"op": op, "B": B, "S": S, "C": C, "G": G, "act": rng.choice(["none", "silu", "gelu"]),
                "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    K = 128 * rng.randint(2, 36)
    R = 8 * rng.randint(1, 16)
    L = rng.randint(1, min(12, 512 // R))
    if op == "block":
        B = _log(rng, 1, 16)
        C = 32 * rng.choice([8, 12, 20, 36, 40, 72])
        return {"op": op, "B": B, "S": _log(rng, 16, 8192 // B), "C": C, "G": 32,
                "act": rng.choice(["none", "silu", "gelu"]), "N": 16 * rng.randint(16, 216), "L": L, "R": R, "Q": B}
    N = 16 * rng.randint(16, 288)
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    # at most the bytes of the largest listed case
    row = (4 if dtype == "fp32" else 2) * (K + 2 * N if op == "adapter" else 2 * K + N)
    M = _log(rng, 1, min(16384, 290_000_000 // row))
    Q = min(M, _log(rng, 1, 96))
    return {"op": op, "M": M, "K": K, "N": N, "L": L, "R": R, "Q": Q, "ragged": rng.random() < 0.6, "dtype": dtype}


# --------------------------------------------------------------------- inputs
def _requests(case, M, gen):
    """Row bounds [Q + 1] and adapter indices [Q] (-1: none) of the requests, int32 on the GPU.

    Ragged: lengths of a random partition (zeros among them), rows behind the last
    request, every eighth request without an adapter.
    """
    Q, L = case["Q"], case["L"]
    index = torch.randint(0, L, (Q,), generator=gen, device="cuda", dtype=torch.int32)
    if case.get("ragged"):
        end = M - M // 16
        cuts = torch.randint(0, end + 1, (max(Q - 1, 0),), generator=gen, device="cuda").sort().values
        bounds = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), end)]).to(torch.int32)
        index[3::8] = -1
    else:
        bounds = (torch.arange(Q + 1, device="cuda") * M // Q).to(torch.int32)
    return bounds, index


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_bwd", "block"):
        B, S, C, G = case["B"], case["S"], case["C"], case["G"]
        dt = DT[case.get("dtype", "bf16")]
        # maps whose groups have means and scales of their own
        x = _randn(gen, B, S, C)
        x.mul_(0.5 + 1.5 * torch.rand(B, 1, C, generator=gen, device="cuda"))
        x.add_(0.7 * _randn(gen, B, 1, C))
        s["x"] = x.to(dt)
        s["gamma"] = 1.0 + 0.2 * _randn(gen, C)
        s["beta"] = 0.2 * _randn(gen, C)
    if op == "norm_bwd":
        s["dy"] = _randn(gen, B, S, C).to(dt)
        s["stats"] = _norm_stats(s["x"], G)          # kept from the forward pass
    if op == "block":
        N = case["N"]
        # the quantized layer: int8 weight codes with per-channel scales, and
        # static activation scales from a calibration pass (values to about 6)
        w = 0.02 * _randn(gen, N, C)
        sw = w.abs().amax(1) / 127
        s["codes"] = (w / sw[:, None]).round().clamp(-127, 127).to(torch.int8)
        s["scales"] = sw[None].contiguous()
        s["s_pos"] = torch.full((1,), 6.0 / 127, device="cuda")
        s["s_neg"] = torch.full((1,), {"none": 6.0, "silu": 0.28, "gelu": 0.17}[case["act"]] / 127, device="cuda")
        M, K, R, L = B * S, C, case["R"], case["L"]
    if op in ("adapter", "adapter_bwd"):
        M, K, N, R, L = case["M"], case["K"], case["N"], case["R"], case["L"]
        dt = DT[case["dtype"]]
        x = _randn(gen, M, K)
        s["x"] = (x * torch.sigmoid(x)).to(dt)       # SiLU features, as the layer's other inputs
    if op in ("adapter", "adapter_bwd", "block"):
        s["a"] = (_randn(gen, L, R, K) / math.sqrt(K)).to(torch.bfloat16)
        s["b"] = (0.3 * _randn(gen, L, N, R) / math.sqrt(R)).to(torch.bfloat16)
        s["scale"] = 0.5 + torch.rand(L, generator=gen, device="cuda")
        s["bounds"], s["index"] = _requests(case, M, gen)
    if op == "adapter":
        s["y"] = _randn(gen, M, N).to(dt)            # the shared projection's output
    if op == "adapter_bwd":
        s["dy"] = _randn(gen, M, N).to(dt)
        hot, _ = _one_hot(s, M)
        h = torch.matmul(s["x"].float(), s["a"].float().view(L * R, K).t()).view(M, L, R)
        s["hidden"] = (h * hot[:, :, None]).sum(1)   # kept from the forward pass
    return s


# ---------------------------------------------------------------- plain forms
def _norm_stats(x, G):
    B, S, C = x.shape
    v = x.float().view(B, S, G, C // G)
    mean = v.mean((1, 3))
    var = (v - mean[:, None, :, None]).square().mean((1, 3))
    return torch.stack([mean, torch.rsqrt(var + EPS)], -1)


def _spread(stats, C):
    """[B, G, 2] -> mean and reciprocal deviation of every channel, [B, 1, C] each."""
    per = stats.repeat_interleave(C // stats.shape[1], 1)
    return per[:, None, :, 0], per[:, None, :, 1]


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _norm(s):
    c = s["case"]
    mean, rstd = _spread(_norm_stats(s["x"], c["G"]), c["C"])
    return _act((s["x"].float() - mean) * rstd * s["gamma"] + s["beta"], c["act"])


def _norm_bwd(s):
    c, x = s["case"], s["x"]
    B, S, C, G = c["B"], c["S"], c["C"], c["G"]
    mean, rstd = _spread(s["stats"], C)
    xhat = (x.float() - mean) * rstd
    dz = s["dy"].float() * _act_slope(xhat * s["gamma"] + s["beta"], c["act"])
    dbeta = dz.sum((0, 1))
    dgamma = (dz * xhat).sum((0, 1))
    dhat = dz * s["gamma"]
    m1 = dhat.view(B, S, G, -1).mean((1, 3)).repeat_interleave(C // G, 1)[:, None]
    m2 = (dhat * xhat).view(B, S, G, -1).mean((1, 3)).repeat_interleave(C // G, 1)[:, None]
    return (rstd * (dhat - m1 - xhat * m2)).to(x.dtype), dgamma, dbeta


def _one_hot(s, M):
    """Which adapter each row has: [M, L] of 0 and 1, and the same times the adapters' scales."""
    L = s["scale"].shape[0]
    rows = torch.arange(M, device="cuda")
    rid = (rows[:, None] >= s["bounds"][None, 1:]).sum(1)
    inside = (rows >= s["bounds"][0]) & (rid < s["index"].shape[0])
    which = torch.where(inside, s["index"][rid.clamp(max=s["index"].shape[0] - 1)], -1)
    hot = (which[:, None] == torch.arange(L, device="cuda")[None]).float()
    return hot, hot * s["scale"]


def _adapter_delta(s, x):
    L, R, K = s["a"].shape
    _, hot = _one_hot(s, x.shape[0])
    h = torch.matmul(x.float(), s["a"].float().view(L * R, K).t()).view(-1, L, R) * hot[:, :, None]
    return torch.matmul(h.view(-1, L * R), s["b"].float().transpose(1, 2).reshape(L * R, -1))


def _adapter_bwd(s):
    L, R, K = s["a"].shape
    M, N = s["dy"].shape
    _, hot = _one_hot(s, M)
    dy, x = s["dy"].float(), s["x"].float()
    b = s["b"].float().transpose(1, 2).reshape(L * R, N)
    u = (torch.matmul(dy, b.t()).view(M, L, R) * hot[:, :, None]).view(M, L * R)
    dx = torch.matmul(u, s["a"].float().view(L * R, K)).to(s["x"].dtype)
    da = torch.matmul(u.t(), x).view(L, R, K)
    h = (s["hidden"][:, None] * hot[:, :, None]).view(M, L * R)
    db = torch.matmul(dy.t(), h).view(N, L, R).transpose(0, 1).contiguous()
    return dx, da, db


def _block(s):
    c = s["case"]
    x16 = _norm(s).to(torch.bfloat16).view(-1, c["C"])
    x = x16.float()
    pos = (x.clamp(min=0) * (1 / s["s_pos"])).round().clamp(0, 127)
    neg = (x.clamp(max=0) * (1 / s["s_neg"])).round().clamp(-127, 0)
    xq = pos * s["s_pos"] + neg * s["s_neg"]
    y = torch.matmul(xq, (s["codes"].float() * s["scales"][0][:, None]).t())
    return (y + _adapter_delta(s, x16)).to(torch.bfloat16), x16


# ------------------------------------------------------------------- one pass
def _layer(s):
    """The handles that a program makes once of its weights: (adapters, quantized weight)."""
    if "handles" not in s:
        import post_quantized_linear_b200 as pq
        qw = None
        if "codes" in s:
            N, K = s["codes"].shape
            qw = pq.QuantizedWeight(8, N, K, (0, K), (0, N), s["codes"], s["scales"])
        s["handles"] = (pq.Adapters(s["a"], s["b"], s["scale"]) if "a" in s else None, qw)
    return s["handles"]


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if own:
        import post_quantized_linear_b200 as pq
        if op == "norm":
            return pq.group_norm_act(s["x"], c["G"], s["gamma"], s["beta"], eps=EPS, act=c["act"])
        if op == "norm_bwd":
            return pq.group_norm_act_backward(s["dy"], s["x"], s["stats"], s["gamma"], s["beta"], act=c["act"])
        adapters, qw = _layer(s)
        if op == "adapter":
            return pq.adapter_add(s["y"], s["x"], adapters, s["bounds"], s["index"])
        if op == "adapter_bwd":
            return pq.adapter_backward(s["dy"], s["x"], s["hidden"], adapters, s["bounds"], s["index"])
        q_pos, q_neg, x16 = pq.quantize_activations_norm(
            s["x"], c["G"], s["gamma"], s["beta"], (0, c["C"]), s["s_pos"], s["s_neg"], eps=EPS,
            act=c["act"], return_y=True)
        # the layer's output in fp32, so that the sum with the adapters' term is rounded once
        y = pq.linear_from_codes(q_pos, q_neg, qw, s["s_pos"], s["s_neg"], out_dtype=torch.float32)
        out = torch.empty_like(y, dtype=torch.bfloat16)
        return pq.adapter_add(y, x16, adapters, s["bounds"], s["index"], out=out), x16
    if op == "norm":
        return _norm(s).to(s["x"].dtype)
    if op == "norm_bwd":
        return _norm_bwd(s)
    if op == "adapter":
        return s["y"].copy_(s["y"].float() + _adapter_delta(s, s["x"]))
    if op == "adapter_bwd":
        return _adapter_bwd(s)
    return _block(s)


# ----------------------------------------------------------------------- work
def work(case):
    c = case
    op = c["op"]
    e = 4 if c.get("dtype") == "fp32" else 2
    if op in ("norm", "norm_bwd"):
        n = c["B"] * c["S"] * c["C"]
        if op == "norm":
            return {"bytes": 2 * n * e + 8 * c["C"], "flops": 8 * n}
        return {"bytes": 3 * n * e + 8 * c["B"] * c["G"] + 16 * c["C"], "flops": 16 * n}
    if op == "block":
        M, K, N = c["B"] * c["S"], c["C"], c["N"]
        rows = M
    else:
        M, K, N = c["M"], c["K"], c["N"]
        # a ragged batch leaves a sixteenth of the rows out, and requests without an adapter
        none = len(range(3, c["Q"], 8)) / c["Q"] if c["ragged"] else 0.0
        rows = (M - M // 16 if c["ragged"] else M) * (1 - none)
    R = c["R"]
    weights = min(c["L"], c["Q"]) * R * (K + N)
    if op == "block":
        return {"bytes": 2 * M * K * 2 + N * K + M * N * 2 + weights * 2,
                "flops": 4 * M * N * K + 2 * rows * R * (K + N)}
    if op == "adapter":
        return {"bytes": rows * (K + 2 * N) * e + weights * 2, "flops": 2 * rows * R * (K + N)}
    return {"bytes": rows * (K + N) * e + M * K * e + rows * R * 4 + weights * 2 + c["L"] * R * (K + N) * 4,
            "flops": 4 * rows * R * (K + N)}


# -------------------------------------------------------------- 64-bit values
def exact(case, seed):
    """The same results from the definitions, in 64 bits: one group, one request at a time."""
    s = prepare(case, seed)
    op = case["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op in ("norm", "norm_bwd", "block"):
        B, S, C = s["x"].shape
        G = case["G"]
        w = C // G
        y = torch.empty(B, S, C, dtype=torch.float64, device="cuda")
        dgamma = torch.zeros(C, dtype=torch.float64, device="cuda")
        dbeta = torch.zeros(C, dtype=torch.float64, device="cuda")
        for i in range(B):
            for g in range(G):
                ch = slice(g * w, (g + 1) * w)
                v, ga, be = d["x"][i, :, ch], d["gamma"][ch], d["beta"][ch]
                if op == "norm_bwd":
                    mean, inv = d["stats"][i, g, 0], d["stats"][i, g, 1]
                else:
                    mean = v.mean()
                    inv = 1 / torch.sqrt(((v - mean) ** 2).mean() + EPS)
                hat = (v - mean) * inv
                z = hat * ga + be
                sig = torch.sigmoid(z)
                phi = torch.special.ndtr(z)
                if op != "norm_bwd":
                    y[i, :, ch] = {"none": z, "silu": z * sig, "gelu": z * phi}[case["act"]]
                    continue
                slope = {"none": torch.ones_like(z), "silu": sig + z * sig * (1 - sig),
                         "gelu": phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)}[case["act"]]
                dz = d["dy"][i, :, ch] * slope
                dbeta[ch] += dz.sum(0)
                dgamma[ch] += (dz * hat).sum(0)
                dh = dz * ga
                y[i, :, ch] = inv * (dh - dh.mean() - hat * (dh * hat).mean())
        if op == "norm":
            return y
        if op == "norm_bwd":
            return y, dgamma, dbeta
    # requests, one after the other
    bounds, index = s["bounds"].tolist(), s["index"].tolist()
    if op == "block":
        x = y.to(torch.bfloat16).double().view(B * S, C)     # the layer's input is stored in bf16
        sp, sn = d["s_pos"], d["s_neg"]
        q = torch.where(x >= 0, torch.round(x / sp).clamp(max=127) * sp, torch.round(x / sn).clamp(min=-127) * sn)
        out = q @ (s["codes"].double() * d["scales"][0][:, None]).t()
    else:
        x = d["x"]
        out = d["y"].clone() if op == "adapter" else torch.zeros_like(x)
    da, db = torch.zeros_like(d["a"]), torch.zeros_like(d["b"])
    for r, l in enumerate(index):
        m = slice(bounds[r], bounds[r + 1])
        if l < 0 or m.start == m.stop:
            continue
        A, Bm, sc = d["a"][l], d["b"][l], d["scale"][l]
        if op == "adapter_bwd":
            u = sc * (d["dy"][m] @ Bm)
            out[m] = u @ A
            da[l] += u.t() @ x[m]
            db[l] += sc * (d["dy"][m].t() @ d["hidden"][m])
        else:
            out[m] += sc * ((x[m] @ A.t()) @ Bm.t())
    if op == "adapter_bwd":
        return out, da, db
    return (out, y.view(B * S, C)) if op == "block" else out
