"""Workloads of the MXFP4 quantisation, the products of two MXFP4 operands (dense and routed to
experts) and the whole expert layer of a few tokens.  Each workload has a plain form in elementary
torch operations and the calls of the library's operators (where `own` is true).

A case names its operator ("op"):
  quantize        mxfp4_quantize / mxfp4_quantize_transposed, with the stored values
  matmul          mxfp4_quantize of the activations, then mxfp4_matmul
  matmul_grad     both gradients of a linear layer: mxfp4_quantize and mxfp4_quantize_transposed
                  along each product's contraction, then mxfp4_matmul
  expert          mxfp4_quantize, then mxfp4_expert_matmul or mxfp4_expert_matmul_swiglu
  layer           mxfp4_moe_layer
"""
import math

import torch

own = False

EPS = 1e-5
DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def listed():
    return [
        # one decoded token's activations (gpt-oss-20b hidden width): latency alone
        {"name": "quantize_one_token", "op": "quantize", "rows": 1, "K": 2880, "x": "bf16", "transposed": False},
        # four experts' gate/up weights of a 32-bit checkpoint, laid into MXFP4 at load time
        {"name": "quantize_weights", "op": "quantize", "rows": 4 * 5760, "K": 2880, "x": "f32", "transposed": False},
        # a training batch's gradient, blocks along the tokens (the contraction of the weight's gradient)
        {"name": "quantize_transposed", "op": "quantize", "rows": 4096, "K": 2880, "x": "bf16", "transposed": True},
        # one decoded token through a linear layer of the gate/up shape
        {"name": "matmul_one_token", "op": "matmul", "M": 1, "N": 5760, "K": 2880, "out": "f32", "bias": True},
        # a prompt of 4096 tokens through the same
        {"name": "matmul_prompt", "op": "matmul", "M": 4096, "N": 5760, "K": 2880, "out": "bf16", "bias": True},
        # a training batch: the gradients of the layer's input and of its weight, from 16-bit tensors
        {"name": "matmul_grad_batch", "op": "matmul_grad", "T": 2048, "N": 5760, "K": 2880},
        # one decoded token through the gate/up projection of its experts and the gated activation
        {"name": "expert_one_token", "op": "expert", "T": 1, "E": 32, "k": 4, "N": 5760, "K": 2880, "swiglu": True,
         "per_slot": False, "zipf": False, "out": "bf16"},
        # a prompt of 4096 tokens through the same
        {"name": "expert_prompt", "op": "expert", "T": 4096, "E": 32, "k": 4, "N": 5760, "K": 2880, "swiglu": True,
         "per_slot": False, "zipf": False, "out": "bf16"},
        # the down projection of a prompt whose experts' loads are far apart, each slot its own input
        {"name": "expert_down_skewed", "op": "expert", "T": 2048, "E": 32, "k": 4, "N": 2880, "K": 2880,
         "swiglu": False, "per_slot": True, "zipf": True, "out": "f32"},
        # one decoded token through a whole layer: norm, router, gate/up, activation, down, combine, residual
        {"name": "layer_one_token", "op": "layer", "T": 1, "E": 32, "k": 4, "H": 2880, "F": 2880, "x": "bf16",
         "norm": True, "residual": True, "y": "bf16"},
        # a small decode batch, the layer's norm on a 32-bit stream, its output added elsewhere
        {"name": "layer_batch", "op": "layer", "T": 8, "E": 32, "k": 4, "H": 2880, "F": 2880, "x": "f32",
         "norm": True, "residual": False, "y": "bf16"},
        # a small odd layer: already normed input, no residual, three of seven experts
        {"name": "layer_odd", "op": "layer", "T": 5, "E": 7, "k": 3, "H": 288, "F": 160, "x": "bf16",
         "norm": False, "residual": False, "y": "bf16"},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul_grad", "expert", "layer"])
    K = 32 * _log_uniform(rng, 1, 180)
    if op == "quantize":
        transposed = rng.random() < 0.5
        if transposed:
            rows = 32 * _log_uniform(rng, 1, 256)
            return {"op": op, "rows": rows, "K": _log_uniform(rng, 1, 5760), "x": rng.choice(["bf16", "f32"]),
                    "transposed": True}
        return {"op": op, "rows": _log_uniform(rng, 1, 4 * 5760 * 2880 // K), "K": K, "x": rng.choice(["bf16", "f32"]),
                "transposed": False}
    if op == "matmul":
        return {"op": op, "M": _log_uniform(rng, 1, 4096), "N": _log_uniform(rng, 1, 5760), "K": K,
                "out": rng.choice(["bf16", "f32"]), "bias": rng.random() < 0.5}
    if op == "matmul_grad":
        return {"op": op, "T": 32 * _log_uniform(rng, 1, 64), "N": 32 * _log_uniform(rng, 1, 180),
                "K": 32 * _log_uniform(rng, 1, 90)}
    E = _log_uniform(rng, 2, 64)
    k = rng.randint(1, min(E, 8))
    if op == "expert":
        swiglu = rng.random() < 0.5
        N = 2 * _log_uniform(rng, 16, 2880) if swiglu else _log_uniform(rng, 16, 5760)
        K = 32 * _log_uniform(rng, 1, 90)
        E = min(E, max(2, 32 * 5760 * 2880 // (N * K)))
        k = min(k, E)
        T = _log_uniform(rng, 1, max(1, min(4096, 4096 * 4 // k)))
        return {"op": op, "T": T, "E": E, "k": k, "N": N, "K": K, "swiglu": swiglu, "per_slot": rng.random() < 0.5,
                "zipf": rng.random() < 0.5, "out": "bf16" if swiglu else rng.choice(["bf16", "f32"])}
    E = min(E, 32) if rng.random() < 0.7 else E
    norm = rng.random() < 0.7
    return {"op": op, "T": rng.randint(1, 8), "E": E, "k": min(k, E, 4), "H": 32 * _log_uniform(rng, 1, 90),
            "F": 32 * _log_uniform(rng, 1, 90), "x": rng.choice(["bf16", "f32"]) if norm else "bf16", "norm": norm,
            "residual": rng.random() < 0.5, "y": "bf16"}


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEVICE)

    def stream(rows, width):
        """Activations: rows of unlike size, a few channels far above the rest."""
        channel = 1.0 + 30.0 * (torch.rand((width,), generator=g, device=DEVICE) < 0.002).float()
        return normal(rows, width) * channel * torch.exp(0.5 * normal(rows, 1))

    def weights(rows, width):
        """MXFP4 codes [*rows, width / 32, 16] and scale bytes of a checkpoint's range."""
        blocks = torch.randint(0, 256, (*rows, width // 32, 16), generator=g, device=DEVICE, dtype=torch.uint8)
        return blocks, torch.randint(118, 124, (*rows, width // 32), generator=g, device=DEVICE, dtype=torch.uint8)

    def empty(shape, dtype):
        return torch.zeros(shape, dtype=dtype, device=DEVICE)

    def packed(rows, width):
        return empty((rows, width // 32, 16), torch.uint8), empty((rows, width // 32), torch.uint8)

    s = dict(case)
    op = case["op"]
    if op == "quantize":
        rows, K = case["rows"], case["K"]
        s["x_in"] = stream(rows, K).to(TYPES[case["x"]])
        out_rows, out_k = (K, rows) if case["transposed"] else (rows, K)
        s["q"] = packed(out_rows, out_k)
        s["values"] = empty((out_rows, out_k), torch.bfloat16)
        return s
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        s["x_in"] = stream(M, K).to(torch.bfloat16)
        s["w"] = weights((N,), K)
        s["b"] = (0.02 * normal(N)).to(torch.bfloat16) if case["bias"] else None
        s["xq"] = packed(M, K)
        s["result"] = empty((M, N), TYPES[case["out"]])
        return s
    if op == "matmul_grad":
        T, N, K = case["T"], case["N"], case["K"]
        s["x_in"] = stream(T, K).to(torch.bfloat16)
        s["dy"] = (0.01 * normal(T, N) * torch.exp(normal(T, 1))).to(torch.bfloat16)
        s["w_in"] = (0.02 * normal(N, K)).to(torch.bfloat16)
        s.update(dyq=packed(T, N), wt=packed(K, N), dyt=packed(N, T), xt=packed(K, T))
        s.update(dx=empty((T, K), torch.bfloat16), dw=empty((N, K), torch.float32))
        return s
    if op == "expert":
        T, E, k, N, K = case["T"], case["E"], case["k"], case["N"], case["K"]
        rows = T * k if case["per_slot"] else T
        s["x_in"] = stream(rows, K).to(torch.bfloat16)
        s["w"] = weights((E, N), K)
        s["b"] = (0.02 * normal(E, N)).to(torch.bfloat16)
        score = torch.rand((T, E), generator=g, device=DEVICE)
        if case["zipf"]:  # drawn without replacement with probabilities that fall as a power of the index
            score = torch.log(torch.arange(1, E + 1, device=DEVICE)) * -1.2 - torch.log(-torch.log(score))
        ids = score.topk(k, dim=1).indices.to(torch.int32)
        flat = ids.reshape(-1)
        s["order"] = torch.sort(flat, stable=True).indices.to(torch.int32)
        counts = torch.bincount(flat, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["counts"] = counts.tolist()
        s["xq"] = packed(rows, K)
        s["result"] = empty((T, k, N // 2 if case["swiglu"] else N), TYPES[case["out"]])
        return s
    T, E, k, H, F = case["T"], case["E"], case["k"], case["H"], case["F"]
    s["x_in"] = stream(T, H).to(TYPES[case["x"]])
    s["w_norm"] = (1.0 + 0.2 * normal(H)).to(torch.bfloat16) if case["norm"] else None
    s["router"] = (normal(E, H) / math.sqrt(H)).to(torch.bfloat16), (0.02 * normal(E)).to(torch.bfloat16)
    s["gu"] = (*weights((E, 2 * F), H), (0.02 * normal(E, 2 * F)).to(torch.bfloat16))
    s["down"] = (*weights((E, H), F), (0.02 * normal(E, H)).to(torch.bfloat16))
    s["result"] = empty((T, H), TYPES[case["y"]])
    s["ids"] = empty((T, k), torch.int32)
    s["gates"] = empty((T, k), torch.float32)
    return s


# ---------------------------------------------------------------- plain forms


def _quantized(x):
    """The values that MXFP4 stores for x [..., K], fp32: blocks of 32 share the power of two that
    brings the largest magnitude into [4, 8), elements go to the nearest of 0 .5 1 1.5 2 3 4 6 (ties
    to the even code, more than 6 to 6)."""
    b = x.float().unflatten(-1, (-1, 32))
    exponent = (torch.frexp(b.abs().amax(-1, keepdim=True)).exponent - 3).clamp(min=-127)
    b = torch.ldexp(b, -exponent)
    a = b.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    return torch.ldexp(torch.copysign(a, b), exponent).flatten(-2)


def _decoded(blocks, scales):
    """fp32 values of MXFP4 codes [..., K / 32, 16] and scale bytes [..., K / 32]."""
    table = torch.tensor(E2M1, device=blocks.device)
    codes = torch.stack([blocks & 15, blocks >> 4], -1).flatten(-2)
    return torch.ldexp(table[codes.int()], scales.int()[..., None] - 127).flatten(-2)


def _swiglu(p):
    gate, up = p[..., 0::2].clamp(max=7.0), p[..., 1::2].clamp(-7.0, 7.0)
    return (up + 1.0) * gate / (1.0 + torch.exp(-1.702 * gate))


def _plain_layer(s):
    T, k = s["T"], s["k"]
    x = s["x_in"].float()
    xn = x
    if s["norm"]:
        xn = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["w_norm"].float()
        xn = xn.to(torch.bfloat16).float()
    logits = xn @ s["router"][0].float().t() + s["router"][1].float()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, top = order.indices[:, :k], order.values[:, :k]
    gates = torch.exp(top - top[:, :1])
    gates = gates / gates.sum(1, keepdim=True)
    rows = []
    for t in range(T):
        e = ids[t]
        p = torch.matmul(_decoded(s["gu"][0][e], s["gu"][1][e]), xn[t]) + s["gu"][2][e].float()
        act = _swiglu(p).to(torch.bfloat16).float()
        out = torch.matmul(_decoded(s["down"][0][e], s["down"][1][e]), act[:, :, None])[:, :, 0]
        rows.append((gates[t, :, None] * (out + s["down"][2][e].float())).sum(0))
    y = torch.stack(rows)
    if s["residual"]:
        y = y + x
    return y.to(s["result"].dtype), ids.to(torch.int32), gates


def _plain(s):
    op = s["op"]
    if op == "quantize":
        x = s["x_in"].t() if s["transposed"] else s["x_in"]
        return _quantized(x.contiguous()).to(torch.bfloat16)
    if op == "matmul":
        y = _quantized(s["x_in"]) @ _decoded(*s["w"]).t()
        if s["b"] is not None:
            y = y + s["b"].float()
        return y.to(s["result"].dtype)
    if op == "matmul_grad":
        dy = s["dy"]
        dx = _quantized(dy) @ _quantized(s["w_in"].t().contiguous()).t()
        dw = _quantized(dy.t().contiguous()) @ _quantized(s["x_in"].t().contiguous()).t()
        return dx.to(torch.bfloat16), dw
    if op == "expert":
        x = _quantized(s["x_in"])
        order = s["order"].long()
        source = order if s["per_slot"] else order // s["k"]
        result = torch.empty_like(s["result"]).flatten(0, 1)
        at = 0
        for e, n in enumerate(s["counts"]):
            if n == 0:
                continue
            p = x[source[at:at + n]] @ _decoded(s["w"][0][e], s["w"][1][e]).t() + s["b"][e].float()
            result[order[at:at + n]] = (_swiglu(p) if s["swiglu"] else p).to(result.dtype)
            at += n
        return result.view_as(s["result"])
    return _plain_layer(s)


# ------------------------------------------------------- the library's calls


def _library(s):
    from mxfp4_mixture_experts_amd import binding as B
    op = s["op"]
    if op == "quantize":
        call = B.mxfp4_quantize_transposed if s["transposed"] else B.mxfp4_quantize
        call(s["x_in"], *s["q"], values=s["values"])
        return s["values"]
    if op == "matmul":
        B.mxfp4_quantize(s["x_in"], *s["xq"])
        B.mxfp4_matmul(*s["xq"], *s["w"], s["M"], s["N"], s["K"], s["result"], bias=s["b"])
        return s["result"]
    if op == "matmul_grad":
        T, N, K = s["T"], s["N"], s["K"]
        B.mxfp4_quantize(s["dy"], *s["dyq"])
        B.mxfp4_quantize_transposed(s["w_in"], *s["wt"])
        B.mxfp4_matmul(*s["dyq"], *s["wt"], T, K, N, s["dx"])
        B.mxfp4_quantize_transposed(s["dy"], *s["dyt"])
        B.mxfp4_quantize_transposed(s["x_in"], *s["xt"])
        B.mxfp4_matmul(*s["dyt"], *s["xt"], N, K, T, s["dw"])
        return s["dx"], s["dw"]
    if op == "expert":
        B.mxfp4_quantize(s["x_in"], *s["xq"])
        call = B.mxfp4_expert_matmul_swiglu if s["swiglu"] else B.mxfp4_expert_matmul
        call(*s["w"], s["b"], s["E"], s["N"], s["K"], *s["xq"], s["per_slot"], s["T"], s["k"], s["offsets"],
             s["order"], s["result"])
        return s["result"]
    if "ws" not in s:  # the workspace that a program keeps beside its buffers, made at the first call
        nbytes = B.mxfp4_moe_layer_workspace_size(s["T"], s["H"], s["E"], s["k"], s["F"])
        s["ws"] = torch.empty((nbytes,), dtype=torch.uint8, device=DEVICE)
    B.mxfp4_moe_layer(s["x_in"], s["T"], s["H"], s["E"], s["k"], s["F"], *s["router"], *s["gu"], *s["down"],
                      s["result"], w_norm=s["w_norm"], eps=EPS, residual=s["residual"], topk_ids=s["ids"],
                      gates=s["gates"], workspace=s["ws"])
    return s["result"], s["ids"], s["gates"]


def run(state):
    return _library(state) if own else _plain(state)


# ----------------------------------------------------------- bytes and exact


def _mx(rows, K):
    return rows * (K // 2 + K // 32)


def work(case):
    """Each input read once, each output written once; of the experts' weights, those of the
    experts that the tokens can reach."""
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["K"]
        return {"bytes": n * (SIZE[case["x"]] + 2) + n // 2 + n // 32, "flops": 4 * n}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + _mx(N, K) + M * N * SIZE[case["out"]] + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    if op == "matmul_grad":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": 2 * (T * K + T * N + N * K) + 2 * T * K + 4 * N * K, "flops": 4 * T * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    used = E * (1.0 - (1.0 - k / E) ** T)  # the experts that T tokens reach on average
    if op == "expert":
        N, K = case["N"], case["K"]
        rows, width = (T * k if case["per_slot"] else T), (N // 2 if case["swiglu"] else N)
        return {"bytes": int(2 * rows * K + used * (_mx(N, K) + 2 * N)) + T * k * width * SIZE[case["out"]] + 8 * T * k,
                "flops": 2 * T * k * N * K}
    H, F = case["H"], case["F"]
    weights = used * (_mx(2 * F, H) + 4 * F + _mx(H, F) + 2 * H)
    return {"bytes": int(weights) + 2 * E * (H + 1) + T * H * (SIZE[case["x"]] + SIZE[case["y"]]) + 8 * T * k + 2 * H,
            "flops": 2 * T * (E * H + k * 3 * F * H)}


def _stored64(x):
    """What MXFP4 stores for x along its last dimension, in 64 bits: the codes counted over the
    midpoints between neighbours (a midpoint goes to the even code)."""
    b = x.double().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))) - 2.0)
    scale = scale.clamp(min=2.0 ** -127)
    a = b.abs() / scale
    code = torch.zeros_like(a, dtype=torch.int64)
    for down in (0.25, 1.25, 2.5, 5.0):
        code += a > down
    for up in (0.75, 1.75, 3.5):
        code += a >= up
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    return (torch.where(b < 0, -1.0, 1.0) * grid[code] * scale).flatten(-2)


def _weights64(blocks, scales):
    low, high = (blocks % 16).long(), (blocks // 16).long()
    code = torch.stack([low, high], dim=-1).flatten(-2)
    level, exponent = code % 2, (code // 2) % 4
    magnitude = torch.where(exponent == 0, level * 0.5, (1.0 + 0.5 * level) * torch.exp2(exponent - 1.0))
    value = torch.where(code >= 8, -magnitude, magnitude).double()
    return (value * torch.exp2(scales.double() - 127.0)[..., None]).flatten(-2)


def _activation64(p):
    gate, up = p[..., 0::2], p[..., 1::2]
    gate = torch.minimum(gate, torch.full_like(gate, 7.0))
    up = torch.maximum(torch.minimum(up, torch.full_like(up, 7.0)), torch.full_like(up, -7.0))
    return gate * torch.sigmoid(1.702 * gate) * (1.0 + up)


def exact(case, seed):
    """The same outputs from the definitions in 64 bits (with the roundings that belong to them:
    what MXFP4 stores, the norm's and the activation's 16 bits)."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _stored64(s["x_in"].t() if case["transposed"] else s["x_in"])
    if op == "matmul":
        y = torch.matmul(_stored64(s["x_in"]), _weights64(*s["w"]).transpose(0, 1))
        return y if s["b"] is None else y + s["b"].double()
    if op == "matmul_grad":
        dy, x, w = s["dy"], s["x_in"], s["w_in"]
        dx = torch.matmul(_stored64(dy), _stored64(w.t()).transpose(0, 1))
        return dx, torch.matmul(_stored64(dy.t()), _stored64(x.t()).transpose(0, 1))
    if op == "expert":
        T, E, k = case["T"], case["E"], case["k"]
        x = _stored64(s["x_in"])
        which = torch.searchsorted(s["offsets"].long(), torch.arange(T * k, device=DEVICE), right=True) - 1
        result = torch.empty((T * k, s["result"].shape[-1]), dtype=torch.float64, device=DEVICE)
        for e in range(E):
            rows = s["order"][which == e].long()
            if rows.numel():
                inputs = x[rows] if case["per_slot"] else x[torch.div(rows, k, rounding_mode="floor")]
                p = torch.matmul(inputs, _weights64(s["w"][0][e], s["w"][1][e]).transpose(0, 1)) + s["b"][e].double()
                result[rows] = _activation64(p) if case["swiglu"] else p
        return result.view(s["result"].shape)
    T, k = case["T"], case["k"]
    x = s["x_in"].double()
    xn = x
    if case["norm"]:
        xn = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * s["w_norm"].double()
        xn = xn.to(torch.bfloat16).double()
    logits = torch.matmul(xn, s["router"][0].double().transpose(0, 1)) + s["router"][1].double()
    ids = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    gates = torch.softmax(logits.gather(1, ids), 1)
    y = x.clone() if case["residual"] else torch.zeros_like(x)
    for t in range(T):
        for slot in range(k):
            e = int(ids[t, slot])
            p = torch.mv(_weights64(s["gu"][0][e], s["gu"][1][e]), xn[t]) + s["gu"][2][e].double()
            act = _activation64(p).to(torch.bfloat16).double()
            out = torch.mv(_weights64(s["down"][0][e], s["down"][1][e]), act) + s["down"][2][e].double()
            y[t] += gates[t, slot] * out
    return y, ids.to(torch.int32), gates
