"""The operators of 8-bit layers with a scale for each block of 128, in plain torch and through the framework.

A layer's products around the latent cache (fused q_a and kv_a, q_b, o, the feed-forward block, fc) on E4M3 operands:
activations have a power-of-two scale per row and 128 inputs, weights an fp32 scale per 128 x 128 block (as checkpoints
bring them).

quantise  rows or a weight matrix to E4M3: the scale is the smallest power of two 2^e, e >= -100, with amax <= 448 * 2^e
          over a row's 128 elements, or over a block of 128 x 128.
matmul    y = x w^T (+ a residual): sum over blocks of sx[block, row] * sw[n / 128, block] * (products of the codes).
ffn       the gated feed-forward block of a layer: rows quantised; silu(x gate^T) * (x up^T), quantised by rows again;
          times down^T, plus the residual stream; bf16, as the next layer takes it.

`own` is set from outside: False computes the plain form, True calls the framework.
"""
import math

import torch

own = False

B = 128
EMIN = -100                     # the smallest scale is 2^EMIN


# --- cases -------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one drafted block's normalised states (fp32, as the norms leave them): latency
        {"name": "quantise_block", "op": "quantise", "rows": 7, "k": 7168, "dtype": "fp32", "weight": False},
        # a prompt's rows before a layer's first product
        {"name": "quantise_prompt", "op": "quantise", "rows": 4000, "k": 7168, "dtype": "bf16", "weight": False},
        # a down projection on its way into the 8-bit format
        {"name": "quantise_weight", "op": "quantise", "rows": 7168, "k": 14336, "dtype": "bf16", "weight": True},
        # the fused q_a and kv_a of a single token: latency
        {"name": "matmul_qkv_a_token", "op": "matmul", "rows": 1, "k": 7168, "n": 2112, "out": "bf16", "add": False},
        # fc over the captured states of one block: weight streaming
        {"name": "matmul_fc_block", "op": "matmul", "rows": 7, "k": 35840, "n": 7168, "out": "fp32", "add": False},
        # odd sizes: ends of every tile and block
        {"name": "matmul_odd", "op": "matmul", "rows": 333, "k": 720, "n": 1808, "out": "bf16", "add": False},
        # q_b of a batch of 32 blocks
        {"name": "matmul_q_b_bs32", "op": "matmul", "rows": 224, "k": 1536, "n": 12288, "out": "bf16", "add": False},
        # o of a prompt, into the residual stream
        {"name": "matmul_o_prompt", "op": "matmul", "rows": 4000, "k": 8192, "n": 7168, "out": "fp32", "add": True},
        # the tiny geometry's feed-forward block: latency of the chain
        {"name": "ffn_tiny", "op": "ffn", "rows": 7, "k": 512, "inter": 1024},
        # one token
        {"name": "ffn_token", "op": "ffn", "rows": 1, "k": 7168, "inter": 14336},
        # a batch of 32 blocks
        {"name": "ffn_bs32", "op": "ffn", "rows": 224, "k": 7168, "inter": 14336},
        # a prompt
        {"name": "ffn_prompt", "op": "ffn", "rows": 2900, "k": 7168, "inter": 14336},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_DIMS = [512, 576, 1024, 1536, 2112, 7168, 8192, 12288, 14336]
_LARGEST = {"quantise": 7168 * 14336, "matmul": 4000 * 8192 * 7168, "ffn": 2900 * 7168 * 14336}


def _dim(rng):
    """A width: one of the framework's geometries, or any multiple of 16."""
    return rng.choice(_DIMS) if rng.random() < 0.6 else 16 * _log(rng, 4, 768)


def draw(rng):
    while True:
        op = rng.choice(["quantise", "matmul", "matmul", "ffn"])
        rows = _log(rng, 1, 5000)
        if op == "quantise":
            c = {"op": op, "rows": rows, "k": _dim(rng), "dtype": rng.choice(["bf16", "fp32"]),
                 "weight": rng.random() < 0.3}
            cost = c["rows"] * c["k"]
        elif op == "matmul":
            add = rng.random() < 0.4
            c = {"op": op, "rows": rows, "k": _dim(rng), "n": _dim(rng),
                 "out": "fp32" if add else rng.choice(["bf16", "fp32"]), "add": add}
            cost = c["rows"] * c["k"] * c["n"]
        else:
            c = {"op": op, "rows": rows, "k": _dim(rng), "inter": _dim(rng)}
            cost = c["rows"] * c["k"] * c["inter"]
        if cost <= _LARGEST[op]:
            return c


def _blocks(n):
    return -(-n // B)


def work(case):
    m, k = case["rows"], case["k"]
    if case["op"] == "quantise":
        size = 2 if case["dtype"] == "bf16" else 4
        scales = (_blocks(m) if case["weight"] else m) * _blocks(k)
        return {"bytes": m * k * (size + 1) + 4 * scales, "flops": 3 * m * k}
    if case["op"] == "matmul":
        n = case["n"]
        out = (2 if case["out"] == "bf16" else 4) + (4 if case["add"] else 0)
        return {"bytes": (m + n) * k + 4 * (m + _blocks(n)) * _blocks(k) + m * n * out, "flops": 2 * m * n * k}
    i = case["inter"]
    return {"bytes": 3 * i * k + 4 * 3 * _blocks(i) * _blocks(k) + m * k * (2 + 4 + 2), "flops": 6 * m * i * k}


# --- inputs ------------------------------------------------------------------------------------------------------
def _weights(n, k, g):
    """Codes [n, k] and fp32 scales of a matrix of N(0, 1/k) elements, scaled by each block's amax / 448."""
    codes = torch.empty(n, k, dtype=torch.uint8, device="cuda")
    scales = torch.empty(_blocks(n), _blocks(k), device="cuda")
    step = B * max(1, (1 << 25) // (B * k))
    for at in range(0, n, step):
        w = torch.randn(min(step, n - at), k, device="cuda", generator=g) / math.sqrt(k)
        p = torch.zeros(_blocks(w.shape[0]) * B, _blocks(k) * B, device="cuda")
        p[:w.shape[0], :k] = w
        s = p.view(-1, B, _blocks(k), B).abs().amax((1, 3)) / 448
        scales[at // B:at // B + s.shape[0]] = s
        q = (p.view(-1, B, _blocks(k), B) / s[:, None, :, None]).clamp(-448, 448).reshape(p.shape)
        codes[at:at + w.shape[0]] = q[:w.shape[0], :k].to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scales


def _activations(m, k, g, dtype):
    """Normalised states: unit normal, some channels some times larger, as trained norms leave them."""
    x = torch.randn(m, k, device="cuda", generator=g)
    wide = torch.rand(k, device="cuda", generator=g) < 0.01
    return (x * torch.where(wide, 12.0, 1.0)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def _row_buffers(m, k):
    return (torch.empty(m, k, dtype=torch.uint8, device="cuda"), torch.empty(_blocks(k), m, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m, k = case["rows"], case["k"]
    if case["op"] == "quantise":
        if case["weight"]:
            x = torch.randn(m, k, device="cuda", generator=g) * 0.02
            x = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
            out = (torch.empty(m, k, dtype=torch.uint8, device="cuda"), torch.empty(_blocks(m), _blocks(k), device="cuda"))
        else:
            x = _activations(m, k, g, case["dtype"])
            out = _row_buffers(m, k)
        return {"case": case, "x": x, "codes": out[0], "scales": out[1]}
    if case["op"] == "matmul":
        n = case["n"]
        w, sw = _weights(n, k, g)
        x, sx = _quantised(_activations(m, k, g, "fp32"))
        state = {"case": case, "w": w, "sw": sw, "x": x, "sx": sx,
                 "y": torch.empty(m, n, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device="cuda")}
        if case["add"]:
            state["residual"] = torch.randn(m, n, device="cuda", generator=g)
        return state
    i = case["inter"]
    state = {"case": case, "x": _activations(m, k, g, "bf16"), "residual": torch.randn(m, k, device="cuda", generator=g),
             "gate": _weights(i, k, g), "up": _weights(i, k, g), "down": _weights(k, i, g),
             "xq": _row_buffers(m, k), "hq": _row_buffers(m, i),
             "y": torch.empty(m, k, dtype=torch.bfloat16, device="cuda")}
    return state


# --- one pass ----------------------------------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return {"quantise": _quantise, "matmul": _matmul, "ffn": _ffn}[state["case"]["op"]](state)


def _run_own(state):
    import mla_block_diffusion_gb300 as M
    case = state["case"]
    if case["op"] == "quantise":
        (M.quantise_weight if case["weight"] else M.quantise_rows)(state["x"], state["codes"], state["scales"])
        return {"codes": state["codes"].view(torch.float8_e4m3fn), "scales": state["scales"]}
    if case["op"] == "matmul":
        if "linear" not in state:
            state["linear"] = M.QLinear(state["w"], state["sw"])
        state["linear"].matmul(state["x"], state["sx"], state["y"], add=state.get("residual"))
        return state["y"]
    if "layers" not in state:
        state["layers"] = (M.QGated(M.QLinear(*state["gate"]), M.QLinear(*state["up"])), M.QLinear(*state["down"]))
    gated, down = state["layers"]
    M.quantise_rows(state["x"], *state["xq"])
    gated.forward(*state["xq"], *state["hq"])
    down.matmul(*state["hq"], state["y"], add=state["residual"])
    return state["y"]


def _exponent(amax):
    """The smallest e >= EMIN with amax <= 448 * 2^e; exact (448 = 0.875 * 2^9)."""
    f, e = torch.frexp(amax)
    e = e - 9 + (f > 0.875).to(e.dtype)
    return torch.where(amax > 0, e, EMIN).clamp(min=EMIN)


def _power(e):
    """2^e in 32 bits, from its exponent field."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _quantised(x, rows=1):
    """Codes and scales by blocks of `rows` x 128; one row: scales [blocks of k, rows of x]."""
    m, k = x.shape
    high, wide = -(-m // rows) * rows, _blocks(k) * B
    p = torch.nn.functional.pad(x.float(), (0, wide - k, 0, high - m)).view(high // rows, rows, wide // B, B)
    e = _exponent(p.abs().amax((1, 3)))
    codes = (p * _power(-e)[:, None, :, None]).reshape(high, wide)[:m, :k].to(torch.float8_e4m3fn).view(torch.uint8)
    scales = _power(e)
    return codes.contiguous(), (scales.t() if rows == 1 else scales).contiguous()


def _quantise(state):
    codes, scales = _quantised(state["x"], B if state["case"]["weight"] else 1)
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}


def _wide_rows(codes, scales):
    """The values of quantised rows, 32 bits."""
    k = codes.shape[1]
    return codes.view(torch.float8_e4m3fn).float() * scales.t().repeat_interleave(B, 1)[:, :k]


def _wide_weights(codes, scales):
    n, k = codes.shape
    return codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(B, 0)[:n].repeat_interleave(B, 1)[:, :k]


def _matmul(state):
    y = _wide_rows(state["x"], state["sx"]) @ _wide_weights(state["w"], state["sw"]).t()
    if "residual" in state:
        y = y + state["residual"]
    return y.to(state["y"].dtype)


def _ffn(state):
    x = _wide_rows(*_quantised(state["x"]))
    gate, up = x @ _wide_weights(*state["gate"]).t(), x @ _wide_weights(*state["up"]).t()
    h = _wide_rows(*_quantised(gate / (1 + torch.exp(-gate)) * up))
    return (h @ _wide_weights(*state["down"]).t() + state["residual"]).to(torch.bfloat16)


# --- the definition in 64 bits -----------------------------------------------------------------------------------
def _e4m3_values():
    """The value of each of the 256 codes: sign, 4 exponent bits of bias 7, 3 fraction bits; 0x7f and 0xff are NaN."""
    v = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v.append(math.nan if c & 127 == 127 else -x if c >= 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _scale64(amax):
    """2^e per element by search: from the exponent of amax / 448, one step up or down where that is off."""
    e = torch.ceil(torch.log2(torch.clamp(amax, min=2.0 ** -300) / 448.0))
    e = torch.where(448.0 * torch.exp2(e) < amax, e + 1, e)
    e = torch.where(448.0 * torch.exp2(e - 1) >= amax, e - 1, e)
    return torch.exp2(torch.clamp(e, min=EMIN))


def _round64(x):
    """To the nearest E4M3 value, halves to the even one."""
    step = torch.exp2(torch.clamp(torch.frexp(x)[1] - 1, -6, 8).double() - 3)
    return torch.round(x / step) * step


def _rows64(x):
    """The values that a quantised row stands for, block by block, and the scales."""
    out, scales = torch.empty_like(x), []
    for at in range(0, x.shape[1], B):
        s = _scale64(x[:, at:at + B].abs().amax(1, keepdim=True))
        out[:, at:at + B] = _round64(x[:, at:at + B] / s) * s
        scales.append(s[:, 0])
    return out, torch.stack(scales)


def exact(case, seed):
    state = prepare(case, seed)
    value = _e4m3_values()
    m, k = case["rows"], case["k"]

    def weights(codes, scales):
        w = value[codes.int()]
        for at in range(0, w.shape[0], B):
            for b in range(scales.shape[1]):
                w[at:at + B, b * B:b * B + B] *= scales[at // B, b].double()
        return w
    if case["op"] == "quantise":
        x = state["x"].double()
        if not case["weight"]:
            v, s = _rows64(x)
            for b in range(s.shape[0]):
                v[:, b * B:b * B + B] /= s[b][:, None]
            return {"codes": v, "scales": s}
        scales = torch.empty(_blocks(m), _blocks(k), dtype=torch.float64, device="cuda")
        for a in range(_blocks(m)):
            rows = x[a * B:a * B + B]
            for b in range(_blocks(k)):
                scales[a, b] = rows[:, b * B:b * B + B].abs().max()
        scales = _scale64(scales)
        for a in range(_blocks(m)):
            for b in range(_blocks(k)):
                x[a * B:a * B + B, b * B:b * B + B] /= scales[a, b]
        return {"codes": _round64(x), "scales": scales}
    if case["op"] == "matmul":
        x = value[state["x"].int()]
        for b in range(_blocks(k)):
            x[:, b * B:b * B + B] *= state["sx"][b].double()[:, None]
        y = torch.einsum("mk,nk->mn", x, weights(state["w"], state["sw"]))
        return y + state["residual"].double() if case["add"] else y
    x = _rows64(state["x"].double())[0]
    gate = torch.einsum("mk,nk->mn", x, weights(*state["gate"]))
    up = torch.einsum("mk,nk->mn", x, weights(*state["up"]))
    h = _rows64(gate * torch.sigmoid(gate) * up)[0]
    return torch.einsum("mk,nk->mn", h, weights(*state["down"])) + state["residual"].double()
