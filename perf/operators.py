"""Workloads of the operators around the expert block: the norms before and after it (with the
combine, the residual scale and the next block's norm) and the routing's balance loss, per-expert
counts and gradients.  Each workload has a plain form in elementary torch operations and the call
of the library's operator (where `own` is true).

A case names its operator ("op") and direction:
  norm, norm_grad                  moe_norm, moe_norm_backward
  combine_norm, combine_norm_grad  moe_combine_norm, moe_combine_norm_backward
  balance                          moe_balance
  route_grad                       moe_route_backward
"""
import math

import torch

own = False

EPS = 1e-5
DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # the block's input norm of one decoded token (gpt-oss-20b hidden width): latency alone
        {"name": "norm_one_token", "op": "norm", "T": 1, "N": 2880, "x": "bf16"},
        # the input norm of a long prompt batch on a residual stream kept in 32 bits
        {"name": "norm_prompt", "op": "norm", "T": 8192, "N": 2880, "x": "f32"},
        # a training batch's input norm, the residual stream's own gradient added
        {"name": "norm_grad_batch", "op": "norm_grad", "T": 8192, "N": 2880, "x": "bf16", "dres": True},
        # an odd width and an odd number of rows: no row but the first starts on 16 bytes
        {"name": "norm_grad_odd", "op": "norm_grad", "T": 1001, "N": 2881, "x": "f32", "dres": False},
        # one decoded token: top-4 combine, residual and the next block's norm
        {"name": "combine_norm_one_token", "op": "combine_norm", "T": 1, "k": 4, "N": 2880, "x": "bf16",
         "proj": "f32", "post": False, "next": True, "unrouted": 0.0, "scale": 1.0},
        # a long prompt batch through combine, output norm, scaled residual and the next norm
        {"name": "combine_norm_prompt", "op": "combine_norm", "T": 8192, "k": 4, "N": 2880, "x": "bf16",
         "proj": "f32", "post": True, "next": True, "unrouted": 0.0, "scale": 0.5},
        # the same in training: the gradients of every input and weight
        {"name": "combine_norm_grad_batch", "op": "combine_norm_grad", "T": 8192, "k": 4, "N": 2880, "x": "bf16",
         "proj": "f32", "post": True, "next": True, "unrouted": 0.0, "scale": 0.5},
        # a ragged batch with unrouted slots (whose rows were never written), bf16 outputs of the experts
        {"name": "combine_norm_grad_ragged", "op": "combine_norm_grad", "T": 777, "k": 3, "N": 1023, "x": "f32",
         "proj": "bf16", "post": True, "next": False, "unrouted": 0.1, "scale": 0.25},
        # one gpt-oss-20b layer's routing of a 4096-token prompt: counts and both losses
        {"name": "balance_prompt", "op": "balance", "T": 4096, "E": 32, "k": 4, "S": 1, "padded": False},
        # packed training sequences over the most experts, with padding behind the last one
        {"name": "balance_packed", "op": "balance", "T": 65536, "E": 512, "k": 8, "S": 37, "padded": True},
        # the gradient of the same two batches' router logits
        {"name": "route_grad_prompt", "op": "route_grad", "T": 4096, "E": 32, "k": 4, "S": 1, "padded": False,
         "out": "f32"},
        {"name": "route_grad_packed", "op": "route_grad", "T": 65536, "E": 512, "k": 8, "S": 37, "padded": True,
         "out": "bf16"},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "combine_norm", "combine_norm_grad", "balance", "route_grad"])
    if op in ("balance", "route_grad"):
        E = _log_uniform(rng, 2, 512)
        T = _log_uniform(rng, 1, 65536)
        case = {"op": op, "T": T, "E": E, "k": rng.randint(1, min(E, 8)), "S": _log_uniform(rng, 1, min(64, T)),
                "padded": rng.random() < 0.5}
        if op == "route_grad":
            case["out"] = rng.choice(["bf16", "f32"])
        return case
    k = rng.randint(1, 8) if op.startswith("combine") else 1
    N = _log_uniform(rng, 32, 8192)
    T = _log_uniform(rng, 1, max(1, min(16384, 8192 * 2880 * (4 if op.startswith("combine") else 1) // (N * k))))
    case = {"op": op, "T": T, "N": N, "x": rng.choice(["bf16", "f32"])}
    if op == "norm_grad":
        case["dres"] = rng.random() < 0.5
    if op.startswith("combine"):
        case.update(k=k, proj=rng.choice(["bf16", "f32"]), post=rng.random() < 0.5, next=rng.random() < 0.7,
                    unrouted=rng.choice([0.0, 0.1]), scale=rng.choice([1.0, 0.5, 0.25]))
    return case


def _sequences(g, T, S, padded):
    """Offsets [S + 1] of S sequences of random lengths (some may be empty) in T tokens; padded: the
    last sequence ends before the tokens do."""
    end = T - int(T * 0.06) if padded else T
    cuts = torch.randint(0, end + 1, (S - 1,), generator=g, device=DEVICE).sort().values
    edges = torch.tensor([0, end], device=DEVICE)
    return torch.cat([edges[:1], cuts, edges[1:]]).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEVICE)

    s = dict(case)
    if case["op"] in ("balance", "route_grad"):
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        # some experts are preferred, a few are masked for a few tokens, a few tokens hold a NaN
        logits = normal(T, E) + normal(E)
        logits[torch.rand((T, E), generator=g, device=DEVICE) < 0.001] = -math.inf
        logits[torch.rand((T,), generator=g, device=DEVICE) < 0.0005, 0] = math.nan
        s["logits"] = logits.to(torch.bfloat16)
        f = s["logits"].float()
        bad = f.isnan().any(1)
        order = torch.sort(f.nan_to_num(0.0, neginf=-1e30), dim=1, descending=True, stable=True).indices[:, :k]
        s["ids"] = torch.where(bad[:, None], torch.full_like(order, -1), order).to(torch.int32).contiguous()
        kept = torch.where(bad[:, None], torch.zeros((), device=DEVICE), f.gather(1, order))
        s["gates"] = torch.where(bad[:, None], torch.zeros((), device=DEVICE), torch.softmax(kept, 1)).contiguous()
        s["seq"] = _sequences(g, T, S, case["padded"])
        s["counts"] = torch.empty((S, E), dtype=torch.int32, device=DEVICE)
        s["tokens"] = torch.empty((S + 2,), dtype=torch.int32, device=DEVICE)
        s["losses"] = torch.empty((2,), dtype=torch.float32, device=DEVICE)
        if case["op"] == "route_grad":
            counts, tokens, _ = _balance(s["logits"], s["ids"], s["seq"])
            s["counts"].copy_(counts)
            s["tokens"].copy_(tokens)
            s["dgates"] = normal(T, k) * 0.1
            s["dlosses"] = torch.tensor([0.01 * T, 0.001 * T], device=DEVICE)
            s["dlogits"] = torch.empty((T, E), dtype=TYPES[case["out"]], device=DEVICE)
        return s
    T, N = case["T"], case["N"]
    x_type = TYPES[case["x"]]
    # a residual stream: rows of unlike size, a few channels far above the rest
    channel = 1.0 + 30.0 * (torch.rand((N,), generator=g, device=DEVICE) < 0.002).float()
    x = (normal(T, N) * channel * torch.exp(0.5 * normal(T, 1))).to(x_type)
    w = (1.0 + 0.2 * normal(N)).to(torch.bfloat16)
    if case["op"] == "norm":
        s.update(x_in=x, w=w, xn=torch.empty((T, N), dtype=torch.bfloat16, device=DEVICE))
        return s
    if case["op"] == "norm_grad":
        s.update(x_in=x, w=w, dxn=normal(T, N).to(torch.bfloat16), dx=torch.empty_like(x),
                 dres_in=normal(T, N).to(x_type) if case["dres"] else None,
                 dw=torch.empty((N,), dtype=torch.float32, device=DEVICE))
        return s
    k = case["k"]
    gates = torch.softmax(normal(T, k), 1)
    lost = torch.rand((T, k), generator=g, device=DEVICE) < case["unrouted"]
    gates[lost] = 0.0
    proj = (0.5 * normal(T, k, N)).to(TYPES[case["proj"]])
    proj[lost] = math.nan  # an unrouted slot's row is never written
    s.update(gates=gates, proj_in=proj, w_post=(1.0 + 0.2 * normal(N)).to(torch.bfloat16) if case["post"] else None,
             w_next=w if case["next"] else None)
    if case["op"] == "combine_norm":
        s.update(x_in=x, x_out=torch.empty_like(x),
                 xn=torch.empty((T, N), dtype=torch.bfloat16, device=DEVICE) if case["next"] else None)
        return s
    s.update(x_stored=x if case["next"] else None, dx_out=normal(T, N).to(x_type),
             dxn=normal(T, N).to(torch.bfloat16) if case["next"] else None,
             dx=torch.empty((T, N), dtype=x_type, device=DEVICE), dproj=torch.empty_like(proj),
             dgates=torch.empty_like(gates),
             dw_post=torch.empty((N,), dtype=torch.float32, device=DEVICE) if case["post"] else None,
             dw_next=torch.empty((N,), dtype=torch.float32, device=DEVICE) if case["next"] else None)
    return s


# ---------------------------------------------------------------- plain forms


def _norm(x, w):
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r * w


def _norm_grad(dy, x, w):
    """Gradients of _norm at x: of x, and the products whose sum over the rows is w's."""
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    unit = x * r
    d = dy * w
    return r * (d - unit * (d * unit).mean(-1, keepdim=True)), dy * unit


def _combine(proj, gates):
    """sum_s gates[t, s] * proj[t, s, :]; a slot with gate 0 adds nothing, whatever its row holds."""
    rows = torch.where(gates[:, :, None] == 0, torch.zeros((), device=proj.device), proj.float())
    return (gates[:, :, None] * rows).sum(1), rows


def _live(logits, ids, seq):
    """The tokens that count, their sequence, their logits (0 where they do not count)."""
    T = logits.shape[0]
    at = torch.arange(T, device=logits.device, dtype=torch.int32)
    which = torch.searchsorted(seq, at, right=True) - 1
    S = seq.numel() - 1
    valid = (ids >= 0) & (ids < logits.shape[1])
    live = (which >= 0) & (which < S) & valid.any(1) & (logits.float().amax(1) != -math.inf)
    f = torch.where(live[:, None], logits.float(), torch.zeros((), device=logits.device))
    return live, which.clamp(0, S - 1), valid & live[:, None], f


def _balance(logits, ids, seq):
    T, E = logits.shape
    S, k = seq.numel() - 1, ids.shape[1]
    live, which, valid, f = _live(logits, ids, seq)
    z = torch.logsumexp(f, 1)
    p = torch.exp(f - z[:, None]) * live[:, None]
    slot = torch.where(valid, which[:, None] * E + ids, S * E).reshape(-1).long()
    counts = torch.zeros(S * E + 1, dtype=torch.int32, device=f.device)
    counts.scatter_add_(0, slot, torch.ones_like(slot, dtype=torch.int32))
    counts = counts[:-1].view(S, E)
    member = (which[None, :] == torch.arange(S, device=f.device)[:, None]) & live[None, :]
    n = member.sum(1)
    mean_p = torch.matmul(member.float(), p) / n.clamp(min=1)[:, None]
    share = counts / (k * n.clamp(min=1))[:, None]
    used = (n > 0).sum()
    balance = (E * (share * mean_p).sum(1)).sum() / used.clamp(min=1)
    total = n.sum()
    z2 = (torch.where(live, z, torch.zeros_like(z)) ** 2).sum() / total.clamp(min=1)
    tokens = torch.cat([n, total[None], used[None]]).to(torch.int32)
    return counts, tokens, torch.stack([balance, z2])


def _route_grad(logits, ids, gates, dgates, seq, counts, tokens, dlosses, out_type):
    T, E = logits.shape
    k = ids.shape[1]
    live, which, valid, f = _live(logits, ids, seq)
    z = torch.logsumexp(f, 1, keepdim=True)
    p = torch.exp(f - z) * live[:, None]
    n = tokens[:-2].float()
    mean = counts.float().sum(1, keepdim=True) / E
    c = (counts - mean) * (E / (k * n.clamp(min=1) ** 2 * tokens[-1].clamp(min=1)))[:, None] * dlosses[0]
    c = c[which]
    d = p * (c - (p * c).sum(1, keepdim=True) + dlosses[1] * (2.0 / tokens[-2].clamp(min=1)) * z)
    q = torch.where(valid, gates, torch.zeros_like(gates))
    dg = torch.where(q != 0, dgates, torch.zeros_like(dgates))
    ds = q * (dg - (q * dg).sum(1, keepdim=True))
    d.scatter_add_(1, ids.clamp(0, E - 1).long(), ds)
    return d.to(out_type)


def _plain(s):
    op = s["op"]
    if op == "norm":
        return _norm(s["x_in"].float(), s["w"].float()).to(torch.bfloat16)
    if op == "norm_grad":
        dx, dw = _norm_grad(s["dxn"].float(), s["x_in"].float(), s["w"].float())
        if s["dres_in"] is not None:
            dx = dx + s["dres_in"].float()
        return dx.to(s["x_in"].dtype), dw.sum(0)
    if op == "combine_norm":
        u, _ = _combine(s["proj_in"], s["gates"])
        if s["w_post"] is not None:
            u = _norm(u, s["w_post"].float())
        x_out = (s["x_in"].float() + s["scale"] * u).to(s["x_in"].dtype)
        if s["w_next"] is None:
            return x_out
        return x_out, _norm(x_out.float(), s["w_next"].float()).to(torch.bfloat16)
    if op == "combine_norm_grad":
        grad = s["dx_out"].float()
        dw_post = dw_next = None
        if s["w_next"] is not None:
            dn, dw_next = _norm_grad(s["dxn"].float(), s["x_stored"].float(), s["w_next"].float())
            grad = grad + dn
            dw_next = dw_next.sum(0)
        h, rows = _combine(s["proj_in"], s["gates"])
        dh = s["scale"] * grad
        if s["w_post"] is not None:
            dh, dw_post = _norm_grad(dh, h, s["w_post"].float())
            dw_post = dw_post.sum(0)
        dproj = (s["gates"][:, :, None] * dh[:, None, :]).to(s["proj_in"].dtype)
        return grad.to(s["dx_out"].dtype), dproj, (dh[:, None, :] * rows).sum(2), dw_post, dw_next
    if op == "balance":
        return _balance(s["logits"], s["ids"], s["seq"])
    return _route_grad(s["logits"], s["ids"], s["gates"], s["dgates"], s["seq"], s["counts"], s["tokens"],
                       s["dlosses"], TYPES[s["out"]])


# ------------------------------------------------------- the library's calls


def _workspace(s, nbytes):
    """The workspace that a program keeps beside its buffers, made at the first call."""
    if "ws" not in s:
        s["ws"] = torch.empty((max(16, nbytes()),), dtype=torch.uint8, device=DEVICE)
    return s["ws"]


def _library(s):
    from mxfp4_mixture_experts_amd import binding as B
    op = s["op"]
    if op == "norm":
        B.moe_norm(s["x_in"], s["w"], s["T"], s["N"], s["xn"], eps=EPS)
        return s["xn"]
    if op == "norm_grad":
        ws = _workspace(s, lambda: B.moe_norm_backward_workspace_size(s["T"], s["N"]))
        B.moe_norm_backward(s["dxn"], s["x_in"], s["w"], s["T"], s["N"], s["dx"], s["dw"], dres=s["dres_in"], eps=EPS,
                            workspace=ws)
        return s["dx"], s["dw"]
    if op == "combine_norm":
        B.moe_combine_norm(s["proj_in"], s["gates"], s["T"], s["k"], s["N"], s["x_in"], s["x_out"],
                           w_post=s["w_post"], scale=s["scale"], w_next=s["w_next"], xn=s["xn"], eps=EPS)
        return s["x_out"] if s["xn"] is None else (s["x_out"], s["xn"])
    if op == "combine_norm_grad":
        ws = _workspace(s, lambda: B.moe_combine_norm_backward_workspace_size(s["T"], s["N"]))
        B.moe_combine_norm_backward(s["dx_out"], s["proj_in"], s["gates"], s["T"], s["k"], s["N"], s["dx"],
                                    dproj=s["dproj"], dgates=s["dgates"], w_post=s["w_post"], dw_post=s["dw_post"],
                                    scale=s["scale"], dxn=s["dxn"], x_out=s["x_stored"], w_next=s["w_next"],
                                    dw_next=s["dw_next"], eps=EPS, workspace=ws)
        return s["dx"], s["dproj"], s["dgates"], s["dw_post"], s["dw_next"]
    if op == "balance":
        ws = _workspace(s, lambda: B.moe_balance_workspace_size(s["T"], s["E"], s["S"]))
        B.moe_balance(s["logits"], s["ids"], s["T"], s["E"], s["k"], s["counts"], s["tokens"], s["losses"],
                      seq_offsets=s["seq"], S=s["S"], workspace=ws)
        return s["counts"], s["tokens"], s["losses"]
    B.moe_route_backward(s["logits"], s["ids"], s["gates"], s["dgates"], s["T"], s["E"], s["k"], s["dlogits"],
                         seq_offsets=s["seq"], S=s["S"], counts=s["counts"], tokens=s["tokens"],
                         dlosses=s["dlosses"])
    return s["dlogits"]


def run(state):
    return _library(state) if own else _plain(state)


# ----------------------------------------------------------- bytes and exact


def work(case):
    """Each input read once, each output written once."""
    op = case["op"]
    if op in ("balance", "route_grad"):
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        if op == "balance":
            return {"bytes": 2 * T * E + 4 * T * k + 4 * (S + 1) + 4 * S * E + 4 * (S + 2) + 8, "flops": 6 * T * E}
        return {"bytes": 2 * T * E + 12 * T * k + 4 * (S + 1) + 4 * S * E + 4 * (S + 2) + 8 + SIZE[case["out"]] * T * E,
                "flops": 9 * T * E}
    T, N, xb = case["T"], case["N"], SIZE[case["x"]]
    if op == "norm":
        return {"bytes": T * N * (xb + 2) + 2 * N, "flops": 4 * T * N}
    if op == "norm_grad":
        return {"bytes": T * N * (2 + 2 * xb + (xb if case["dres"] else 0)) + 6 * N, "flops": 12 * T * N}
    k, pb = case["k"], SIZE[case["proj"]]
    weights = 2 * N * (case["post"] + case["next"])
    if op == "combine_norm":
        return {"bytes": T * k * N * pb + 4 * T * k + 2 * T * N * xb + (2 * T * N if case["next"] else 0) + weights,
                "flops": T * N * (2 * k + 4 * case["post"] + 2 + 4 * case["next"])}
    return {"bytes": 2 * T * k * N * pb + 8 * T * k + 2 * T * N * xb + (T * N * (2 + xb) if case["next"] else 0)
            + 3 * weights, "flops": T * N * (5 * k + 12 * case["post"] + 12 * case["next"] + 2)}


def exact(case, seed):
    """The same outputs from the definitions in 64 bits; the gradients come from differentiating the
    64-bit forward formulas."""
    s = prepare(case, seed)
    op = case["op"]

    def wide(t):
        return None if t is None else t.double()

    def rms(x, w):
        return x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w

    if op == "norm":
        return rms(wide(s["x_in"]), wide(s["w"]))
    if op == "norm_grad":
        x, w = wide(s["x_in"]).requires_grad_(), wide(s["w"]).requires_grad_()
        dx, dw = torch.autograd.grad((rms(x, w) * wide(s["dxn"])).sum(), (x, w))
        return dx if s["dres_in"] is None else dx + wide(s["dres_in"]), dw
    if op.startswith("combine"):
        gates = wide(s["gates"])
        rows = torch.nan_to_num(wide(s["proj_in"]), nan=0.0)
        w_post, w_next = wide(s["w_post"]), wide(s["w_next"])

        def block(rows, gates, w_post):
            h = (gates[:, :, None] * rows).sum(1)
            return h if w_post is None else rms(h, w_post)

        if op == "combine_norm":
            x_out = wide(s["x_in"]) + case["scale"] * block(rows, gates, w_post)
            if w_next is None:
                return x_out
            return x_out, rms(x_out.to(s["x_in"].dtype).double(), w_next)
        grad, dw_next, dw_post = wide(s["dx_out"]), None, None
        if w_next is not None:
            x_out = wide(s["x_stored"]).requires_grad_()
            w_next.requires_grad_()
            dn, dw_next = torch.autograd.grad((rms(x_out, w_next) * wide(s["dxn"])).sum(), (x_out, w_next))
            grad = grad + dn
        leaves = [rows.requires_grad_(), gates.requires_grad_()]
        if w_post is not None:
            leaves.append(w_post.requires_grad_())
        got = torch.autograd.grad((case["scale"] * block(rows, gates, w_post) * grad).sum(), leaves)
        routed = s["gates"] != 0
        if w_post is not None:
            dw_post = got[2]
        return grad, got[0], got[1] * routed, dw_post, dw_next
    logits, ids, seq = s["logits"], s["ids"].long(), s["seq"].tolist()
    T, E, k = case["T"], case["E"], case["k"]
    inside = torch.zeros(T, dtype=torch.bool, device=DEVICE)
    inside[seq[0]:seq[-1]] = True
    live = inside & (ids >= 0).any(1) & (logits != -math.inf).any(1)
    f = torch.where(live[:, None], wide(logits), torch.zeros((), dtype=torch.float64, device=DEVICE))
    f.requires_grad_()
    p, z = torch.softmax(f, 1), torch.logsumexp(f, 1)
    onehot = torch.zeros((T, E), dtype=torch.float64, device=DEVICE)
    onehot.scatter_add_(1, ids.clamp(min=0), ((ids >= 0) & live[:, None]).double())
    parts = []
    for a, b in zip(seq[:-1], seq[1:]):
        n = int(live[a:b].sum())
        if n:
            fraction = onehot[a:b].sum(0) / (k * n)
            parts.append(E * (fraction * (p[a:b] * live[a:b, None]).sum(0) / n).sum())
    zero = (f * 0.0).sum()
    balance = torch.stack(parts).mean() if parts else zero
    z2 = (z.square() * live).sum() / live.sum().clamp(min=1)
    if op == "balance":
        return None, None, torch.stack([balance, z2]).detach()
    dl = wide(s["dlosses"])
    d = torch.autograd.grad(dl[0] * balance + dl[1] * z2 + zero, f)[0]
    q, dg = torch.where(live[:, None], wide(s["gates"]), torch.zeros_like(wide(s["gates"]))), wide(s["dgates"])
    d.scatter_add_(1, ids.clamp(min=0), q * (dg - (q * dg).sum(1, keepdim=True)))
    return d
