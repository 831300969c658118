"""Cases of the 8-bit linear-layer operators: what each computes, on which sizes, and what it has to move.

The operators are those of a linear layer, and of the gated activation between two of them, that keep their
inputs in 8 bits from the forward pass to the backward pass:

  checkpoint   rows of activations -> int8 codes and one power-of-two scale per row, and back
  matmul       y = diag(sx) (Xq Wq^T) diag(sw) + bias, from the codes of both
  input_grad   dX = dY diag(sw) Wq
  weight_grad  dW = dY^T diag(sx) Xq, from the codes that the forward pass kept; dbias = column sums of dY
  swiglu       h = silu(gate) * up, kept as codes, and (dgate, dup) from the codes of gate and up

run() computes them in 32 bits with elementary torch operations, or, where `own` is true, with this package's calls.
"""
import math

import torch

own = False

MAX_FLOPS = 2 * 8192 * 16384 * 4096      # the largest listed product
MAX_ELEMENTS = 16384 * 8192              # the largest listed array of activations


def listed():
    return [
        # a small layer's fp32 activations, rows that are not a multiple of anything
        {"name": "checkpoint ragged", "op": "checkpoint", "tokens": 1537, "dim": 1001, "dtype": "float32"},
        # one layer's activations of a training batch
        {"name": "checkpoint layer", "op": "checkpoint", "tokens": 16384, "dim": 8192, "dtype": "bfloat16"},
        # one new token through a square projection: latency, and the weights' bytes
        {"name": "matmul one token", "op": "matmul", "tokens": 1, "n": 4096, "k": 4096, "bias": False, "dtype": "bfloat16"},
        # a batch of requests, one new token each, through an up projection
        {"name": "matmul decode batch", "op": "matmul", "tokens": 48, "n": 11000, "k": 4096, "bias": True, "dtype": "bfloat16"},
        # one prompt of odd length through odd widths, fp32 results
        {"name": "matmul ragged prompt", "op": "matmul", "tokens": 777, "n": 4104, "k": 2050, "bias": True, "dtype": "float32"},
        # a training batch through an up projection
        {"name": "matmul training", "op": "matmul", "tokens": 8192, "n": 16384, "k": 4096, "bias": False, "dtype": "bfloat16"},
        # a small layer's backward pass at odd sizes
        {"name": "input grad ragged", "op": "input_grad", "tokens": 1000, "n": 1531, "k": 2052, "dtype": "bfloat16"},
        # a training batch through a square projection, backwards
        {"name": "input grad training", "op": "input_grad", "tokens": 8192, "n": 4096, "k": 4096, "dtype": "bfloat16"},
        # a small layer's weights at odd sizes, with its bias
        {"name": "weight grad ragged", "op": "weight_grad", "tokens": 1001, "n": 776, "k": 1505, "bias": True, "dtype": "bfloat16"},
        # a training batch's fp32 gradient of a down projection
        {"name": "weight grad training", "op": "weight_grad", "tokens": 8192, "n": 4096, "k": 16384, "bias": False, "dtype": "float32"},
        # a few tokens through a narrow gated block
        {"name": "swiglu small", "op": "swiglu", "tokens": 33, "dim": 1408},
        # a training batch through a wide gated block
        {"name": "swiglu training", "op": "swiglu", "tokens": 8192, "dim": 16384},
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, its logarithm uniform: half of them multiples of 64, the others any number."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        v = (v + 63) // 64 * 64
    v = max(lo, min(hi, v))
    return 3071 if v == 3072 else v


def draw(rng):
    op = rng.choice(("checkpoint", "matmul", "matmul", "input_grad", "weight_grad", "swiglu"))
    if op in ("checkpoint", "swiglu"):
        dim = _size(rng, 64, 16384)
        tokens = _size(rng, 1, 16384)
        tokens = max(1, min(tokens, MAX_ELEMENTS // dim))
        case = {"op": op, "tokens": tokens, "dim": dim}
        if op == "checkpoint":
            case["dtype"] = rng.choice(("bfloat16", "float32"))
        return case
    n, k = _size(rng, 64, 16384), _size(rng, 64, 16384)
    tokens = _size(rng, 1 if op == "matmul" else 64, 8192)
    tokens = max(1, min(tokens, MAX_FLOPS // (2 * n * k)))
    case = {"op": op, "tokens": tokens, "n": n, "k": k, "dtype": rng.choice(("bfloat16", "float32"))}
    if op != "input_grad":
        case["bias"] = rng.random() < 0.5
    return case


# --------------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, tokens, dim):
    """N(0, 1) with a few channels an order of magnitude above the others, as activations have."""
    x = _normal(gen, tokens, dim)
    loud = torch.rand(dim, generator=gen, device="cuda") < 0.002
    x[:, loud] *= 10.0
    return x


def _scale(a):
    """The smallest power of two s >= 2^-126 with a / s < 127.5; 0 for a = 0."""
    _, e = torch.frexp(a)
    s = torch.ldexp(torch.ones_like(a), (e - 7).clamp(min=-126))
    s = torch.where(a >= 127.5 * s, 2 * s, s)
    return torch.where(a == 0, torch.zeros_like(s), s)


def _encode(x):
    """int8 codes and one scale per row, in 32 bits."""
    s = _scale(x.abs().amax(dim=-1))
    q = torch.round(x / torch.where(s == 0, torch.ones_like(s), s).unsqueeze(-1))
    return q.to(torch.int8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    state = {"case": case}
    op, tokens = case["op"], case["tokens"]
    if op == "checkpoint":
        state["x"] = _activations(gen, tokens, case["dim"]).to(getattr(torch, case["dtype"]))
    elif op == "swiglu":
        state["gate_up"] = _normal(gen, tokens, 2 * case["dim"]).to(torch.bfloat16)
        state["dh"] = (1e-3 * _normal(gen, tokens, case["dim"])).to(torch.bfloat16)
    else:
        n, k = case["n"], case["k"]
        if op in ("matmul", "weight_grad"):
            state["x_codes"], state["x_scale"] = _encode(_activations(gen, tokens, k).to(torch.bfloat16).float())
        if op in ("matmul", "input_grad"):
            state["w_codes"], state["w_scale"] = _encode(_normal(gen, n, k) / math.sqrt(k))
        if op == "matmul":
            state["bias"] = 0.1 * _normal(gen, n) if case["bias"] else None
        else:
            state["dy"] = (1e-3 * _normal(gen, tokens, n)).to(torch.bfloat16)
    return state


# ----------------------------------------------------------------- the passes

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "checkpoint":
        codes, scale = _encode(state["x"].float())
        return {"restored": (codes.float() * scale.unsqueeze(1)).to(torch.bfloat16), "scale": scale}
    if op == "swiglu":
        dim = case["dim"]
        gu = state["gate_up"].float()
        gate, up = gu[:, :dim], gu[:, dim:]
        h_codes, h_scale = _encode(gate / (1 + torch.exp(-gate)) * up)
        gate_codes, gate_scale = _encode(gate)
        up_codes, up_scale = _encode(up)
        gate = gate_codes.float() * gate_scale.unsqueeze(1)
        up = up_codes.float() * up_scale.unsqueeze(1)
        dh = state["dh"].float()
        sig = 1 / (1 + torch.exp(-gate))
        dgate = dh * up * sig * (1 + gate * (1 - sig))
        dup = dh * gate * sig
        return {"h": (h_codes.float() * h_scale.unsqueeze(1)).to(torch.bfloat16), "h_scale": h_scale,
                "saved_scale": torch.stack((gate_scale, up_scale), dim=1),
                "dgate_up": torch.cat((dgate, dup), dim=1).to(torch.bfloat16)}
    out = getattr(torch, case["dtype"])
    if op == "matmul":
        y = state["x_codes"].float() @ state["w_codes"].float().t()
        y = y * state["x_scale"].unsqueeze(1) * state["w_scale"]
        if state["bias"] is not None:
            y = y + state["bias"]
        return {"y": y.to(out)}
    dy = state["dy"].float()
    if op == "input_grad":
        return {"dx": (dy @ (state["w_codes"].float() * state["w_scale"].unsqueeze(1))).to(out)}
    got = {"dw": (dy.t() @ (state["x_codes"].float() * state["x_scale"].unsqueeze(1))).to(out)}
    if case["bias"]:
        got["dbias"] = dy.sum(dim=0)
    return got


def _run_own(state):
    import embedding_communication_codecs_gb300 as q
    case = state["case"]
    op = case["op"]
    if op == "checkpoint":
        codes, scale = q.rowwise_int8(state["x"])
        return {"restored": q.rowwise_int8_dequant(codes, scale, dtype=torch.bfloat16), "scale": scale}
    if op == "swiglu":
        h_codes, h_scale, saved_codes, saved_scale = q.swiglu_encode(state["gate_up"])
        return {"h": q.rowwise_int8_dequant(h_codes, h_scale, dtype=torch.bfloat16), "h_scale": h_scale,
                "saved_scale": saved_scale,
                "dgate_up": q.swiglu_backward(state["dh"], saved_codes, saved_scale)}
    out = getattr(torch, case["dtype"])
    if op == "matmul":
        return {"y": q.int8_matmul(state["x_codes"], state["x_scale"], state["w_codes"], state["w_scale"],
                                   bias=state["bias"], dtype=out)}
    if op == "input_grad":
        return {"dx": q.int8_input_grad(state["dy"], state["w_codes"], state["w_scale"], dtype=out)}
    dw, dbias = q.int8_weight_grad(state["dy"], state["x_codes"], state["x_scale"], dtype=out,
                                   with_bias=case["bias"])
    return {"dw": dw, "dbias": dbias} if case["bias"] else {"dw": dw}


# ------------------------------------------------------------------ its work

def work(case):
    op, t = case["op"], case["tokens"]
    size = {"bfloat16": 2, "float32": 4}.get(case.get("dtype"))
    if op == "checkpoint":
        # saved by one call and restored by another, much later: the codes are written and read
        e = t * case["dim"]
        return {"bytes": e * (size + 1) + 4 * t + e * (1 + 2) + 4 * t, "flops": 2 * e}
    if op == "swiglu":
        # forward: gate and up in, their codes and h's out; backward: the codes and dh in, two gradients
        # out; and h's codes back to values
        e = t * case["dim"]
        return {"bytes": e * (4 + 2 + 1) + 12 * t + e * (2 + 2 + 4) + 8 * t + e * (1 + 2) + 4 * t, "flops": 30 * e}
    n, k = case["n"], case["k"]
    if op == "matmul":
        moved = t * k + 4 * t + n * k + 4 * n + (4 * n if case["bias"] else 0) + t * n * size
    elif op == "input_grad":
        moved = 2 * t * n + n * k + 4 * n + t * k * size
    else:
        moved = 2 * t * n + t * k + 4 * t + n * k * size + (4 * n if case["bias"] else 0)
    return {"bytes": moved, "flops": 2 * t * n * k}


# ------------------------------------------------------- the same in 64 bits

def _rows64(x):
    """codes * scale of the rows of a 64-bit array, and the scales, by logarithms instead of bit fields."""
    top = x.abs().max(dim=-1).values
    live = top > 0
    e = torch.floor(torch.log2(torch.where(live, top, torch.ones_like(top)))) - 6
    unit = torch.exp2(e)
    unit = torch.where(top / unit >= 128, unit * 2, unit)      # a logarithm that came out one low
    unit = torch.where(top / unit < 64, unit / 2, unit)        # or one high
    unit = torch.where(top / unit >= 127.5, unit * 2, unit)
    unit = unit.clamp(min=2.0 ** -126)
    values = torch.round(x / unit[..., None]) * unit[..., None]
    return torch.where(live[..., None], values, torch.zeros_like(values)), torch.where(live, unit, torch.zeros_like(unit))


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "checkpoint":
        values, scale = _rows64(state["x"].double())
        return {"restored": values, "scale": scale}
    if op == "swiglu":
        gate, up = state["gate_up"].double().chunk(2, dim=1)
        h, h_scale = _rows64(gate * torch.sigmoid(gate) * up)
        g, g_scale = _rows64(gate)
        u, u_scale = _rows64(up)
        sig = torch.sigmoid(g)
        dh = state["dh"].double()
        return {"h": h, "h_scale": h_scale, "saved_scale": torch.stack((g_scale, u_scale), dim=1),
                "dgate_up": torch.cat((dh * u * (sig + g * sig * (1 - sig)), dh * g * sig), dim=1)}
    if op == "matmul":
        x = state["x_codes"].double() * state["x_scale"].double()[:, None]
        w = state["w_codes"].double() * state["w_scale"].double()[:, None]
        y = torch.einsum("tk,nk->tn", x, w)
        return {"y": y if state["bias"] is None else y + state["bias"].double()}
    dy = state["dy"].double()
    if op == "input_grad":
        return {"dx": torch.einsum("tn,nk->tk", dy, state["w_codes"].double() * state["w_scale"].double()[:, None])}
    got = {"dw": torch.einsum("tn,tk->nk", dy, state["x_codes"].double() * state["x_scale"].double()[:, None])}
    if case["bias"]:
        got["dbias"] = torch.einsum("tn->n", dy)
    return got
