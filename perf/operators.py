"""Cases of the transformer operators around the pruned layers: RMS norm with
the residual's addition and an 8-bit output, its backward pass, the block-scaled
8-bit quantiser, and the block-scaled 8-bit Linear layer.

``run`` computes a case either in plain torch operations (``own`` false) or by
the library's entry points (``own`` true); ``exact`` computes it in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
BLOCK = 128
SMALLEST_SCALE = 2.0 ** -100
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}


def listed():
    return [
        # one token of a decode loop enters a layer: residual stream updated, 8-bit input of the next product
        {"name": "norm_token", "op": "norm", "T": 1, "D": 4096, "type": "f16", "residual": True, "out": "q"},
        # a prompt of 8192 tokens, the same step
        {"name": "norm_prompt", "op": "norm", "T": 8192, "D": 4096, "type": "bf16", "residual": True, "out": "q"},
        # training forward on a ragged batch and a width that no vector load divides: 16-bit output, 1/rms kept
        {"name": "norm_ragged", "op": "norm", "T": 1013, "D": 1001, "type": "f16", "residual": False, "out": "y"},
        # training backward at a full batch, gradient of the residual branch added
        {"name": "norm_grad", "op": "norm_grad", "T": 8192, "D": 4096, "type": "bf16", "residual": True},
        # backward in 32 bits on a ragged batch of a narrow model
        {"name": "norm_grad_ragged", "op": "norm_grad", "T": 517, "D": 1023, "type": "f32", "residual": False},
        # a training step's activations: groups of 128 along both axes, for the product and for the weight gradient
        {"name": "quant_tokens", "op": "quant", "R": 8192, "C": 4096, "type": "bf16", "block": 1, "fp8": "e4m3"},
        # a feed-forward weight after an optimizer step: 128 x 128 blocks, plain and transposed
        {"name": "quant_weight", "op": "quant", "R": 11008, "C": 4096, "type": "f16", "block": 128, "fp8": "e4m3"},
        # decode, one token through a 4096 x 4096 projection
        {"name": "linear_token", "op": "linear", "T": 1, "R": 4096, "K": 4096, "block": 128, "x": "e4m3", "type": "f16",
         "act": "none"},
        # decode of 16 sequences through the wide feed-forward projection, bias and GELU
        {"name": "linear_decode", "op": "linear", "T": 16, "R": 11008, "K": 4096, "block": 128, "x": "e4m3",
         "type": "bf16", "act": "gelu"},
        # a short ragged prompt through a small layer of odd sizes, 32-bit output
        {"name": "linear_ragged", "op": "linear", "T": 777, "R": 1000, "K": 1041, "block": 128, "x": "e4m3",
         "type": "f32", "act": "relu"},
        # weight gradient of a 4096 x 1024 layer over 8192 tokens: gradient in e5m2, both sides in groups along the tokens
        {"name": "linear_wgrad", "op": "linear", "T": 4096, "R": 1024, "K": 8192, "block": 1, "x": "e5m2", "type": "f32",
         "act": "none"},
        # a prompt of 8192 tokens through the wide feed-forward projection
        {"name": "linear_prompt", "op": "linear", "T": 8192, "R": 11008, "K": 4096, "block": 128, "x": "e4m3",
         "type": "bf16", "act": "none"},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], evenly over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "quant", "linear", "linear", "linear"])
    if op == "norm":
        return {"op": op, "T": _spread(rng, 1, 8192), "D": _spread(rng, 64, 11008),
                "type": rng.choice(["f16", "bf16", "f32"]), "residual": rng.random() < 0.7, "out": rng.choice(["q", "y", "yq"])}
    if op == "norm_grad":
        return {"op": op, "T": _spread(rng, 1, 8192), "D": _spread(rng, 64, 11008),
                "type": rng.choice(["f16", "bf16", "f32"]), "residual": rng.random() < 0.7}
    if op == "quant":
        return {"op": op, "R": _spread(rng, 1, 11008), "C": _spread(rng, 64, 11008),
                "type": rng.choice(["f16", "bf16", "f32"]), "block": rng.choice([1, 128]), "fp8": rng.choice(["e4m3", "e5m2"])}
    T, R, K = _spread(rng, 1, 8192), _spread(rng, 64, 11008), _spread(rng, 64, 8192)
    return {"op": op, "T": min(T, 8192 * 11008 * 4096 // (R * K)), "R": R, "K": K,
            "block": rng.choice([128, 128, 1]), "x": rng.choice(["e4m3", "e4m3", "e5m2"]),
            "type": rng.choice(["f16", "bf16", "f32"]), "act": rng.choice(["none", "relu", "gelu"])}


# ------------------------------------------------------------------ inputs


def _groups(n):
    return -(-n // BLOCK)


def _blocks(x, rows):
    """x (R x C) zero-padded and cut into blocks of rows x 128: (R/rows, rows, C/128, 128)."""
    R, C = x.shape
    x = torch.nn.functional.pad(x, (0, -C % BLOCK, 0, -R % rows))
    return x.view(x.shape[0] // rows, rows, -1, BLOCK)


def _quantized(x, rows, fp8):
    """The 8-bit form of an fp32 x: (q, s), one scale for each rows x 128 block."""
    b = _blocks(x, rows)
    s = (b.abs().amax((1, 3)) / FP8_MAX[fp8]).clamp_min(SMALLEST_SCALE)
    q = (b / s[:, None, :, None]).clamp(-FP8_MAX[fp8], FP8_MAX[fp8])
    return q.reshape(b.shape[0] * rows, -1)[: x.shape[0], : x.shape[1]].to(fp8), s


def _widened(q, s, rows):
    """The fp32 values that (q, s) stands for."""
    R, K = q.shape
    b = _blocks(q.float(), rows) * s[:, None, :, None]
    return b.reshape(b.shape[0] * rows, -1)[:R, :K]


def _pitched(q):
    """q with rows 16-byte aligned, as the tensor memory copies want them."""
    R, C = q.shape
    buf = torch.zeros((R, -(-C // 16) * 16), dtype=torch.uint8, device=q.device)
    buf[:, :C] = q.view(torch.uint8)
    return buf.view(q.dtype)[:, :C]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def activations(T, D):
        # a few features are much larger than the rest, as in trained models
        return normal(T, D) * (1.0 + 15.0 * (torch.rand(D, generator=g, device=dev) < 0.005).float())

    st = dict(case)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        T, D, dt = case["T"], case["D"], DTYPES[case["type"]]
        st["w"] = (1.0 + 0.1 * normal(D)).to(dt)
        if op == "norm":
            st["x"] = activations(T, D).to(dt)
            if case["residual"]:
                st["res"] = activations(T, D).to(dt)
                st["h"] = torch.empty_like(st["x"])
            if "y" in case["out"]:
                st["y"] = torch.empty_like(st["x"])
                st["rstd"] = torch.empty(T, device=dev)
            if "q" in case["out"]:
                st["q"] = torch.empty((T, D), dtype=torch.float8_e4m3fn, device=dev)
                st["s"] = torch.empty((T, _groups(D)), device=dev)
        else:
            st["hs"] = activations(T, D).to(dt)
            st["rstd"] = torch.rsqrt(st["hs"].float().square().mean(-1) + EPS)
            st["dy"] = (0.01 * normal(T, D)).to(dt)
            if case["residual"]:
                st["dres"] = (0.01 * normal(T, D)).to(dt)
            st["dh"] = torch.empty_like(st["hs"])
            st["dw"] = torch.empty(D, device=dev)
    elif op == "quant":
        R, C, rows, fp8 = case["R"], case["C"], case["block"], FP8[case["fp8"]]
        st["x"] = (activations(R, C) if rows == 1 else 0.02 * normal(R, C)).to(DTYPES[case["type"]])
        st["q"] = _pitched(torch.zeros((R, C), dtype=torch.uint8, device=dev).view(fp8))
        st["qt"] = _pitched(torch.zeros((C, R), dtype=torch.uint8, device=dev).view(fp8))
        st["s"] = torch.empty((-(-R // rows), _groups(C)), device=dev)
        st["st"] = torch.empty((-(-C // rows), _groups(R)), device=dev)
    else:
        T, R, K, rows = case["T"], case["R"], case["K"], case["block"]
        x = activations(T, K) if case["x"] == "e4m3" else 0.01 * normal(T, K)
        w = 0.02 * normal(R, K) if rows == 128 else activations(R, K)
        xq, st["xs"] = _quantized(x, 1, FP8[case["x"]])
        wq, st["ws"] = _quantized(w, rows, torch.float8_e4m3fn)
        st["xq"], st["wq"] = _pitched(xq), _pitched(wq)
        st["bias"] = normal(R).to(DTYPES[case["type"]]) if case["act"] != "none" else None
        st["y"] = torch.empty((T, R), dtype=DTYPES[case["type"]], device=dev)
    return st


# ------------------------------------------------------------------ one pass


def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from structured_sparse_matmul_gb300 import vnm
    op = st["op"]
    if op == "norm":
        out = {k: st[k] for k in ("h", "y", "rstd", "q", "s") if k in st}
        vnm.vnm_rmsnorm(st["x"], st["w"], EPS, residual=st.get("res"), h=st.get("h"), y=st.get("y"), rstd=st.get("rstd"),
                        q=st.get("q"), q_scale=st.get("s"))
        return out
    if op == "norm_grad":
        vnm.vnm_rmsnorm_backward(st["dy"], st["hs"], st["w"], st["rstd"], st["dh"], st["dw"], dresidual=st.get("dres"))
        return {"dh": st["dh"], "dw": st["dw"]}
    if op == "quant":
        vnm.vnm_fp8_quantize(st["x"], st["q"], st["s"], st["qt"], st["st"], block_rows=st["block"])
        return {"q": st["q"], "s": st["s"], "qt": st["qt"], "st": st["st"]}
    act = {"none": vnm.VNM_ACT_NONE, "relu": vnm.VNM_ACT_RELU, "gelu": vnm.VNM_ACT_GELU}[st["act"]]
    vnm.vnm_fp8_linear(st["xq"], st["xs"], st["wq"], st["ws"], st["y"], bias=st["bias"], act=act)
    return st["y"]


def _run_plain(st):
    op = st["op"]
    if op == "norm":
        out, h = {}, st["x"]
        if st["residual"]:
            h = out["h"] = (st["x"].float() + st["res"].float()).to(st["x"].dtype)
        h = h.float()
        rstd = torch.rsqrt(h.square().mean(-1) + EPS)
        y = h * rstd[:, None] * st["w"].float()
        if "y" in st["out"]:
            out["y"], out["rstd"] = y.to(st["x"].dtype), rstd
        if "q" in st["out"]:
            out["q"], out["s"] = _quantized(y, 1, torch.float8_e4m3fn)
        return out
    if op == "norm_grad":
        dy, h, rstd = st["dy"].float(), st["hs"].float(), st["rstd"][:, None]
        g = dy * st["w"].float()
        dh = rstd * (g - h * rstd.square() * (g * h).mean(-1, keepdim=True))
        if st["residual"]:
            dh = dh + st["dres"].float()
        return {"dh": dh.to(st["hs"].dtype), "dw": (dy * h * rstd).sum(0)}
    if op == "quant":
        x, fp8 = st["x"].float(), FP8[st["fp8"]]
        q, s = _quantized(x, st["block"], fp8)
        qt, s_t = _quantized(x.t().contiguous(), st["block"], fp8)
        return {"q": q, "s": s, "qt": qt, "st": s_t}
    y = _widened(st["xq"], st["xs"], 1) @ _widened(st["wq"], st["ws"], st["block"]).t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    if st["act"] == "relu":
        y = y.clamp_min(0.0)
    elif st["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    return y.to(st["y"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "linear":
        T, R, K = case["T"], case["R"], case["K"]
        e = torch.empty((), dtype=DTYPES[case["type"]]).element_size()
        scales = 4 * _groups(K) * (T + -(-R // case["block"]))
        return {"bytes": T * K + R * K + scales + e * (T * R + (R if case["act"] != "none" else 0)), "flops": 2 * T * R * K}
    e = torch.empty((), dtype=DTYPES[case["type"]]).element_size()
    if op == "quant":
        R, C, rows = case["R"], case["C"], case["block"]
        return {"bytes": R * C * (e + 2) + 4 * (-(-R // rows) * _groups(C) + -(-C // rows) * _groups(R)), "flops": 4 * R * C}
    T, D = case["T"], case["D"]
    if op == "norm":
        b = e * (T * D + D) + (2 * e * T * D if case["residual"] else 0)
        b += (e * T * D + 4 * T if "y" in case["out"] else 0) + (T * D + 4 * T * _groups(D) if "q" in case["out"] else 0)
        return {"bytes": b, "flops": 6 * T * D}
    return {"bytes": e * (T * D * (4 if case["residual"] else 3) + D) + 4 * (T + D), "flops": 10 * T * D}


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]

    def f64(t):
        return t.double()

    def scaled(v, rows, top):
        """v divided by its blocks' scales, not rounded to 8 bits; and the scales."""
        R, C = v.shape
        s = torch.zeros((-(-R // rows), _groups(C)), dtype=torch.float64, device=v.device)
        wide = torch.empty_like(v)
        for j in range(_groups(C)):
            part = v[:, j * BLOCK:(j + 1) * BLOCK].abs().max(1).values
            part = torch.cat([part, part.new_zeros(-R % rows)]).view(-1, rows).max(1).values
            s[:, j] = (part / top).clamp(min=SMALLEST_SCALE)
            wide[:, j * BLOCK:(j + 1) * BLOCK] = v[:, j * BLOCK:(j + 1) * BLOCK] / \
                s[:, j].repeat_interleave(rows)[:R].unsqueeze(1)
        return wide, s

    if op == "norm":
        out, h = {}, f64(st["x"])
        if st["residual"]:
            h = out["h"] = f64((h + f64(st["res"])).to(st["x"].dtype))
        ms = torch.einsum("td,td->t", h, h) / st["D"]
        y = torch.einsum("td,t,d->td", h, 1.0 / torch.sqrt(ms + EPS), f64(st["w"]))
        if "y" in st["out"]:
            out["y"], out["rstd"] = y, 1.0 / torch.sqrt(ms + EPS)
        if "q" in st["out"]:
            out["q"], out["s"] = scaled(y, 1, 448.0)
        return out
    if op == "norm_grad":
        dy, h, w, r = f64(st["dy"]), f64(st["hs"]), f64(st["w"]), f64(st["rstd"])
        dot = torch.einsum("td,d,td->t", dy, w, h) / st["D"]
        dh = r[:, None] * dy * w - (r ** 3 * dot)[:, None] * h
        if st["residual"]:
            dh += f64(st["dres"])
        return {"dh": dh, "dw": torch.einsum("td,td,t->d", dy, h, r)}
    if op == "quant":
        top = 448.0 if st["fp8"] == "e4m3" else 57344.0
        q, s = scaled(f64(st["x"]), st["block"], top)
        qt, s_t = scaled(f64(st["x"]).t().contiguous(), st["block"], top)
        return {"q": q, "s": s, "qt": qt, "st": s_t}
    y = torch.zeros((st["T"], st["R"]), dtype=torch.float64, device=st["y"].device)
    for j in range(_groups(st["K"])):
        k = slice(j * BLOCK, (j + 1) * BLOCK)
        w_scale = f64(st["ws"][:, j]).repeat_interleave(st["block"])[: st["R"]]
        y += (f64(st["xq"][:, k].float()) @ f64(st["wq"][:, k].float()).t()) * torch.outer(f64(st["xs"][:, j]), w_scale)
    if st["bias"] is not None:
        y += f64(st["bias"])
    if st["act"] == "relu":
        y = torch.where(y > 0, y, torch.zeros_like(y))
    elif st["act"] == "gelu":
        y = y * 0.5 * torch.erfc(-y / math.sqrt(2.0))
    return y
