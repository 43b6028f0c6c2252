"""Cases of the dense 16-bit layers of a feed-forward block: the product with
bias, activation and residual and its gradients' products; the gated pair of
projections with its activation checkpoints in 16 or 8 bits; and its backward pass.

``run`` computes a case either in plain torch operations (``own`` false) or by
the library's entry points (``own`` true); ``exact`` computes it in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

GROUP = 128
SMALLEST_SCALE = 2.0 ** -100
LARGEST = 448.0  # of e4m3
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # decode, one token: the down projection of a 4096-wide layer, added to the residual stream
        {"name": "dense_token", "op": "dense", "T": 1, "R": 4096, "K": 11008, "type": "f16", "out": "f16", "layout": "plain",
         "bias": False, "act": "none", "residual": True},
        # a short ragged prompt through a small layer of odd sizes, everything in the epilogue
        {"name": "dense_ragged", "op": "dense", "T": 517, "R": 1001, "K": 1041, "type": "bf16", "out": "bf16",
         "layout": "plain", "bias": True, "act": "gelu", "residual": True},
        # a prompt of 8192 tokens through the down projection, added to the residual stream
        {"name": "dense_prompt", "op": "dense", "T": 8192, "R": 4096, "K": 11008, "type": "bf16", "out": "bf16",
         "layout": "plain", "bias": False, "act": "none", "residual": True},
        # gradient of the input of that projection over a ragged batch: dY . W, W as it is stored
        {"name": "dense_input_grad", "op": "dense", "T": 1013, "R": 11008, "K": 4096, "type": "f16", "out": "f16",
         "layout": "input", "bias": False, "act": "none", "residual": False},
        # weight gradient of a 4096 x 1024 layer over 8192 tokens, added to a 32-bit gradient
        {"name": "dense_weight_grad", "op": "dense", "T": 4096, "R": 1024, "K": 8192, "type": "bf16", "out": "f32",
         "layout": "weight", "bias": False, "act": "none", "residual": True},
        # decode, one token through the gated pair of projections
        {"name": "gated_token", "op": "gated", "T": 1, "K": 4096, "F": 11008, "type": "f16", "act": "silu", "keep": "none"},
        # decode of 16 sequences
        {"name": "gated_decode", "op": "gated", "T": 16, "K": 4096, "F": 11008, "type": "bf16", "act": "silu", "keep": "none"},
        # training forward on a ragged batch of a small model, the projections kept in 16 bits
        {"name": "gated_ragged", "op": "gated", "T": 333, "K": 1023, "F": 1001, "type": "f16", "act": "gelu", "keep": "16"},
        # training forward at a full batch, the projections kept in 8 bits
        {"name": "gated_train", "op": "gated", "T": 8192, "K": 4096, "F": 11008, "type": "bf16", "act": "silu", "keep": "8"},
        # its backward pass from the 8-bit checkpoint, with the hidden activations for the next layer's weight gradient
        {"name": "gated_grad", "op": "gated_grad", "T": 8192, "K": 4096, "F": 11008, "type": "bf16", "act": "silu",
         "keep": "8", "hidden": True},
        # backward of a small layer over one short batch, from 16-bit checkpoints
        {"name": "gated_grad_small", "op": "gated_grad", "T": 1024, "K": 1024, "F": 4096, "type": "bf16", "act": "gelu",
         "keep": "16", "hidden": False},
        # backward on the ragged batch
        {"name": "gated_grad_ragged", "op": "gated_grad", "T": 333, "K": 1023, "F": 1001, "type": "f16", "act": "gelu",
         "keep": "16", "hidden": True},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], evenly over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dense", "dense", "gated", "gated", "gated_grad"])
    kind = rng.choice(["f16", "bf16"])
    if op == "dense":
        layout = rng.choice(["plain", "plain", "input", "weight"])
        plain = layout == "plain"
        R, K = _spread(rng, 64, 11008), _spread(rng, 64, 11008)
        return {"op": op, "T": min(_spread(rng, 1, 8192), 8192 * 4096 * 11008 // (R * K)), "R": R, "K": K, "type": kind,
                "out": rng.choice([kind, kind, "f32"]), "layout": layout, "bias": plain and rng.random() < 0.5,
                "act": rng.choice(["none", "relu", "gelu", "silu"]) if plain else "none", "residual": rng.random() < 0.5}
    case = {"op": op, "T": _spread(rng, 1, 8192), "K": _spread(rng, 64, 4096), "F": _spread(rng, 64, 11008), "type": kind,
            "act": rng.choice(["silu", "silu", "gelu", "relu"])}
    if op == "gated":
        return {**case, "keep": rng.choice(["none", "16", "8"])}
    return {**case, "keep": rng.choice(["16", "8"]), "hidden": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs


def _groups(n):
    return -(-n // GROUP)


def _blocks(x):
    """x (T x F) zero-padded and cut into groups of 128 columns: (T, F/128, 128)."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % GROUP)).view(x.shape[0], -1, GROUP)


def _quantized(x):
    """The 8-bit form of an fp32 x: (q, s), one scale for each 128 columns of a row."""
    b = _blocks(x)
    s = (b.abs().amax(2) / LARGEST).clamp_min(SMALLEST_SCALE)
    q = (b / s[:, :, None]).clamp(-LARGEST, LARGEST)
    return q.reshape(x.shape[0], -1)[:, : x.shape[1]].to(torch.float8_e4m3fn), s


def _widened(q, s):
    """The fp32 values that (q, s) stands for; q itself in 32 bits without scales."""
    if s is None:
        return q.float()
    return (_blocks(q.float()) * s[:, :, None]).reshape(q.shape[0], -1)[:, : q.shape[1]]


def _pitched(x):
    """x (16-bit) with rows 16-byte aligned, as the tensor memory copies want them."""
    R, C = x.shape
    buf = torch.zeros((R, -(-C // 8) * 8), dtype=x.dtype, device=x.device)
    buf[:, :C] = x
    return buf[:, :C]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def activations(T, D):
        # a few features are much larger than the rest, as in trained models
        return normal(T, D) * (1.0 + 15.0 * (torch.rand(D, generator=g, device=dev) < 0.005).float())

    st, dt = dict(case), DTYPES[case["type"]]
    if case["op"] == "dense":
        T, R, K, layout, out = case["T"], case["R"], case["K"], case["layout"], DTYPES[case["out"]]
        if layout == "weight":  # dY (tokens x T) and X (tokens x R), as the forward pass left them
            st["x"], st["w"] = _pitched((0.01 * normal(K, T)).to(dt)).t(), _pitched(activations(K, R).to(dt)).t()
        elif layout == "input":  # dY, and the weights as they are stored (K x R)
            st["x"], st["w"] = _pitched((0.01 * normal(T, K)).to(dt)), _pitched((0.02 * normal(K, R)).to(dt)).t()
        else:
            st["x"], st["w"] = _pitched(activations(T, K).to(dt)), _pitched((0.02 * normal(R, K)).to(dt))
        st["b"] = normal(R).to(dt) if case["bias"] else None
        st["r"] = normal(T, R).to(out) if case["residual"] else None
        st["y"] = torch.empty((T, R), dtype=out, device=dev)
        return st
    T, K, F = case["T"], case["K"], case["F"]
    st["x"] = _pitched(activations(T, K).to(dt))
    st["wg"], st["wu"] = _pitched((0.02 * normal(F, K)).to(dt)), _pitched((0.02 * normal(F, K)).to(dt))
    if case["op"] == "gated":
        st["y"] = _pitched(torch.zeros((T, F), dtype=dt, device=dev))
        for k in ("g", "u"):
            if case["keep"] == "16":
                st[k] = torch.empty((T, F), dtype=dt, device=dev)
            elif case["keep"] == "8":
                st[k] = torch.empty((T, F), dtype=torch.float8_e4m3fn, device=dev)
                st[k + "s"] = torch.empty((T, _groups(F)), device=dev)
        return st
    for k in ("g", "u"):  # of the size that the products have
        v = normal(T, F) * (0.02 * math.sqrt(K) * 1.5)
        if case["keep"] == "8":
            st[k], st[k + "s"] = _quantized(v)
        else:
            st[k] = v.to(dt)
    st["dy"] = _pitched((0.01 * normal(T, F)).to(dt))
    st["dx"] = torch.empty((T, K), dtype=dt, device=dev)
    st["dwg"], st["dwu"] = torch.empty((F, K), dtype=dt, device=dev), torch.empty((F, K), dtype=dt, device=dev)
    st["h"] = _pitched(torch.zeros((T, F), dtype=dt, device=dev)) if case["hidden"] else None
    return st


# ------------------------------------------------------------------ one pass


def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from structured_sparse_matmul_gb300 import vnm
    act = {"none": vnm.VNM_ACT_NONE, "relu": vnm.VNM_ACT_RELU, "gelu": vnm.VNM_ACT_GELU, "silu": vnm.VNM_ACT_SILU}[st["act"]]
    if st["op"] == "dense":
        vnm.vnm_dense_linear(st["x"], st["w"], st["y"], bias=st["b"], act=act, residual=st["r"])
        return st["y"]
    kept = {k: st[k] for k in ("g", "u") if k in st}
    kept.update({k + "_scale": st[k + "s"] for k in ("g", "u") if k + "s" in st})
    if st["op"] == "gated":
        vnm.vnm_gated_linear(st["x"], st["wg"], st["wu"], st["y"], act=act, **kept)
        return {k: st[k] for k in ("y", "g", "u", "gs", "us") if k in st}
    vnm.vnm_gated_linear_backward(st["dy"], st["x"], st["wg"], st["wu"], act=act, dx=st["dx"], dwg=st["dwg"], dwu=st["dwu"],
                                  h=st["h"], **kept)
    return {k: st[k] for k in ("dx", "dwg", "dwu", "h") if st[k] is not None}


def _activated(z, act):
    """(act(z), act'(z))"""
    if act == "relu":
        return z.clamp_min(0.0), (z > 0).float()
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    return z, torch.ones_like(z)


def _run_plain(st):
    x, dt = st["x"].float(), st["x"].dtype
    if st["op"] == "dense":
        y = x @ st["w"].float().t()
        if st["b"] is not None:
            y = y + st["b"].float()
        y = _activated(y, st["act"])[0]
        if st["r"] is not None:
            y = y + st["r"].float()
        return y.to(st["y"].dtype)
    wg, wu = st["wg"].float(), st["wu"].float()
    if st["op"] == "gated":
        g, u = x @ wg.t(), x @ wu.t()
        out = {"y": (_activated(g, st["act"])[0] * u).to(dt)}
        if st["keep"] == "16":
            out["g"], out["u"] = g.to(dt), u.to(dt)
        elif st["keep"] == "8":
            (out["g"], out["gs"]), (out["u"], out["us"]) = _quantized(g), _quantized(u)
        return out
    g, u, dy = _widened(st["g"], st.get("gs")), _widened(st["u"], st.get("us")), st["dy"].float()
    a, slope = _activated(g, st["act"])
    dg, du = dy * u * slope, dy * a
    out = {"dx": (dg @ wg + du @ wu).to(dt), "dwg": (dg.t() @ x).to(dt), "dwu": (du.t() @ x).to(dt)}
    if st["h"] is not None:
        out["h"] = (a * u).to(dt)
    return out


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    T, K = case["T"], case["K"]
    if case["op"] == "dense":
        R, e = case["R"], 4 if case["out"] == "f32" else 2
        b = 2 * (T * K + R * K + (R if case["bias"] else 0)) + e * T * R * (2 if case["residual"] else 1)
        return {"bytes": b, "flops": 2 * T * R * K}
    F = case["F"]
    kept = {"none": 0, "16": 4 * T * F, "8": 2 * T * (F + 4 * _groups(F))}[case["keep"]]  # both projections
    if case["op"] == "gated":
        return {"bytes": 2 * (T * K + 2 * F * K + T * F) + kept, "flops": 4 * T * F * K}
    b = 2 * (T * F + 2 * T * K + 4 * F * K + (T * F if case["hidden"] else 0)) + kept
    return {"bytes": b, "flops": 8 * T * F * K}


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    st = prepare(case, seed)

    def f64(t):
        return t.double()

    def gate(z):
        if case["act"] == "relu":
            return torch.where(z > 0, z, torch.zeros_like(z))
        if case["act"] == "gelu":
            return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * torch.sigmoid(z) if case["act"] == "silu" else z

    if case["op"] == "dense":
        y = torch.einsum("tk,rk->tr", f64(st["x"]), f64(st["w"]))
        if case["bias"]:
            y += f64(st["b"])
        y = gate(y)
        return y + f64(st["r"]) if case["residual"] else y

    def scaled(v):
        """v divided by its groups' scales, not rounded to 8 bits; and the scales."""
        s = torch.zeros((v.shape[0], _groups(v.shape[1])), dtype=torch.float64, device=v.device)
        wide = torch.empty_like(v)
        for j in range(s.shape[1]):
            part = v[:, j * GROUP:(j + 1) * GROUP]
            s[:, j] = (part.abs().max(1).values / LARGEST).clamp(min=SMALLEST_SCALE)
            wide[:, j * GROUP:(j + 1) * GROUP] = part / s[:, j, None]
        return wide, s

    if case["op"] == "gated":
        g, u = (torch.einsum("tk,fk->tf", f64(st["x"]), f64(st[w])) for w in ("wg", "wu"))
        out = {"y": gate(g) * u}
        if case["keep"] == "16":
            out["g"], out["u"] = g, u
        elif case["keep"] == "8":
            (out["g"], out["gs"]), (out["u"], out["us"]) = scaled(g), scaled(u)
        return out

    def kept(k):
        v = f64(st[k].float())
        return v if case["keep"] == "16" else v * f64(st[k + "s"]).repeat_interleave(GROUP, 1)[:, : case["F"]]

    g, u, dy = kept("g"), kept("u"), f64(st["dy"])
    if case["act"] == "relu":
        slope = (g > 0).double()
    elif case["act"] == "gelu":
        slope = 0.5 * torch.erfc(-g / math.sqrt(2.0)) + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)
    else:
        slope = torch.sigmoid(g) + g * torch.sigmoid(g) * torch.sigmoid(-g)
    dg, du = dy * u * slope, dy * gate(g)
    out = {"dx": torch.einsum("tf,fk->tk", dg, f64(st["wg"])) + torch.einsum("tf,fk->tk", du, f64(st["wu"])),
           "dwg": torch.einsum("tf,tk->fk", dg, f64(st["x"])), "dwu": torch.einsum("tf,tk->fk", du, f64(st["x"]))}
    if case["hidden"]:
        out["h"] = gate(g) * u
    return out
