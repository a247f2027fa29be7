"""Cases, plain forms and calls of what stands around the MoE layer in a model, and of its form for a few tokens.

Operators (T tokens of width d; the layer has E experts of width F, k of them for a token):

  norm           n = x r(x) w with r(x) = 1 / sqrt(mean(x^2) + eps): the norm before a block
  norm_grad      its gradient, with the gradient that reaches x beside the norm added
  residual       out = res + s sigmoid(gate) drop(p)(v), v = y r(y) post_w or y: the norm behind a block, its gate,
                 dropout and residual scale; with the norm before the next block, n = out r(out) next_w
  residual_grad  its gradient, every input's
  dropout        out_i = keep_i x_i / (1 - p), keep_i from a counter-based generator; the same call on a gradient is
                 the gradient
  decode         a whole pre-norm MoE block for a few tokens: norm, router, experts, combine, residual

Dropout's generator is Philox 4x32 with 10 rounds: elements 8 b .. 8 b + 7 take the 16-bit halves, low half first, of
the four words for counter {b, step} and key {seed} (64 bits each, low word first), and an element is kept where its
half is at least floor(65536 p + 1/2) = t; 1 / (1 - p) is 65536 / (65536 - t).
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6
#: Most elements of a residual case, and of one of dropout, and most weights of one matrix of all experts.
_MOST_TD, _MOST_DROP, _MOST_W = 4096 * 4096, 8192 * 14336, 8 * 4096 * 14336
#: Most bytes of x in a decode case.
_MOST_X = 131072


def listed():
    """Sizes of the workloads this repository measures (its Mixtral-shaped, 64-expert, capacity and tiny shapes)."""
    mix = dict(d=4096, E=8, k=2, F=14336)
    cap = dict(d=2048, E=64, k=6, F=1408)
    row = dict(dtype="bf16", post=True, next=True, gate="none", p=0.0, scale=1.0)
    dec = dict(op="decode", dtype="bf16", weights="dtype", blocked=True, norm=True, res=True, given=False)
    return [
        # a decode step's rows before its router
        dict(name="norm_t32", op="norm", T=32, d=4096, dtype="bf16"),
        # the pre-norm of a training micro-batch
        dict(name="norm_grad_t4096", op="norm_grad", T=4096, d=2048, dtype="bf16"),
        # one token between two blocks: latency
        dict(row, name="residual_t1", op="residual", T=1, d=3584),
        # a training micro-batch with everything between two blocks
        dict(row, name="residual_t4096", op="residual", T=4096, d=4096, gate="token", p=0.1, scale=0.5),
        dict(row, name="residual_grad_t4096", op="residual_grad", T=4096, d=4096, gate="token", p=0.1, scale=0.5),
        # fp32, the smallest layer
        dict(row, name="residual_grad_tiny_f32", op="residual_grad", T=64, d=128, dtype="f32", gate="full", p=0.25),
        # dropout of a block's output in a small batch, and of the experts' SwiGLU intermediate in a large one
        dict(name="dropout_t512", op="dropout", n=512 * 4096, dtype="bf16", p=0.1),
        dict(name="dropout_h_t4096", op="dropout", n=8192 * 14336, dtype="bf16", p=0.1),
        # one sequence being answered
        dict(mix, **dec, name="decode_t1", T=1),
        # a few sequences, weights in 8 bits
        dict(mix, **dict(dec, weights="e4m3"), name="decode_t8_fp8", T=8),
        # many small experts, weights as they are stored
        dict(cap, **dict(dec, blocked=False), name="decode_e64_t4", T=4),
        # fp32, the smallest layer: launches count
        dict(d=128, E=8, k=2, F=256, **dict(dec, dtype="f32", blocked=False), name="decode_tiny_f32", T=8),
    ]


def draw(rng):
    """One more case of the same ranges: rows of one to 8192 tokens and widths of 64 to 8192; dropout of one element to
    the largest listed; one to 16 tokens through layers of two to 64 experts."""
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm_grad", "residual", "residual_grad", "residual_grad", "dropout", "decode", "decode",
                     "decode"])
    dtype = "bf16" if rng.random() < 0.7 else "f32"
    p = rng.choice([0.0, 0.1, 0.5, round(rng.uniform(0.01, 0.9), 3)])
    if op == "dropout":
        return dict(op=op, n=spread(1, _MOST_DROP // 2), dtype=dtype, p=p)
    if op != "decode":
        d = 64 * spread(1, 128)
        T = spread(1, min(8192, _MOST_TD // 2 // d))
        if op in ("norm", "norm_grad"):
            return dict(op=op, T=T, d=d, dtype=dtype)
        return dict(op=op, T=T, d=d, dtype=dtype, post=rng.random() < 0.7, next=rng.random() < 0.7,
                    gate=rng.choice(["none", "token", "full"]), p=p, scale=rng.choice([1.0, 0.22, -0.5]))
    E = spread(2, 64)
    k = rng.randint(1, min(E, 8))
    d, F = 64 * spread(2, 64), 64 * spread(2, 224)
    while E * d * F > _MOST_W / 2:
        F = max(64, F // 128 * 64)
    T = spread(1, min(16, _MOST_X // (d * (2 if dtype == "bf16" else 4))))
    weights = "e4m3" if dtype == "bf16" and rng.random() < 0.3 else "dtype"
    return dict(op=op, T=T, d=d, E=E, k=k, F=F, dtype=dtype, weights=weights, blocked=rng.random() < 0.5,
                norm=rng.random() < 0.7, res=rng.random() < 0.7, given=rng.random() < 0.3)


def work(case):
    """Bytes (inputs read once, outputs written once) and operations of one pass."""
    c = case
    eb = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "dropout":
        return {"bytes": 2.0 * c["n"] * eb, "flops": 1.0 * c["n"]}
    T, d = float(c["T"]), c["d"]
    tok = T * d * eb
    if c["op"] == "norm":
        return {"bytes": 2 * tok + d * eb, "flops": 4 * T * d}
    if c["op"] == "norm_grad":
        return {"bytes": 4 * tok + 2 * d * eb, "flops": 10 * T * d}
    if c["op"] in ("residual", "residual_grad"):
        gate = {"none": 0.0, "token": T * eb, "full": tok}[c["gate"]]
        vecs = (c["post"] + c["next"]) * d * eb
        if c["op"] == "residual":
            return {"bytes": (3 + c["next"]) * tok + gate + vecs, "flops": 12 * T * d}
        return {"bytes": (4 + 2 * c["next"]) * tok + 2 * gate + 2 * vecs, "flops": 30 * T * d}
    E, k, F = c["E"], c["k"], c["F"]
    active = E * (1.0 - (1.0 - k / E) ** c["T"])  # experts that at least one of T even draws takes
    wb = 1 if c["weights"] == "e4m3" else eb
    return {"bytes": 3 * active * d * F * wb + (2 + c["res"]) * tok + (0 if c["given"] else E * d * eb),
            "flops": 6 * T * k * d * F + 2 * T * E * d}


# ---- inputs -----------------------------------------------------------------


def _randn(gen, dtype, *shape, std=1.0, mean=0.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda") * std + mean)
    return out


def _blocked16(w):
    """The storage order in which each group of 16 rows holds 64-byte pieces of its rows one after another."""
    e, n, m = w.shape
    per = 64 // w.element_size()
    return w.view(e, n // 16, 16, m // per, per).transpose(2, 3).contiguous().view(e, n, m)


def _e4m3(w):
    """Codes and one fp32 scale for each row; expert by expert, so that the fp32 copies stay small."""
    codes = torch.empty(w.shape, dtype=torch.uint8, device="cuda")
    scale = torch.empty(w.shape[:2], dtype=torch.float32, device="cuda")
    for e in range(w.shape[0]):
        v = w[e].float()
        scale[e] = v.abs().amax(1).clamp_(min=1e-12) / 448.0
        codes[e] = (v / scale[e].unsqueeze(1)).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scale


def prepare(case, seed):
    """Inputs and buffers a program has in hand: activations, weights, gradients from behind, the generator's state."""
    c = dict(case)
    dt = _TYPES[c["dtype"]]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 29)
    s = {"case": c}
    if c["op"] == "dropout" or c.get("p"):
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=gen, device="cuda")  # seed and step
    if c["op"] == "dropout":
        s["x"] = _randn(gen, dt, c["n"])
    elif c["op"] == "decode":
        _prepare_decode(s, gen, dt)
    else:
        T, d = c["T"], c["d"]
        if c["op"] in ("norm", "norm_grad"):
            s["x"], s["w"] = _randn(gen, dt, T, d), _randn(gen, dt, d, std=0.2, mean=1.0)
            if c["op"] == "norm_grad":
                s["dn"], s["dres"] = _randn(gen, dt, T, d), _randn(gen, dt, T, d)
        else:
            s["y"] = _randn(gen, dt, T, d, std=0.5)
            s["post"] = _randn(gen, dt, d, std=0.2, mean=1.0) if c["post"] else None
            s["next"] = _randn(gen, dt, d, std=0.2, mean=1.0) if c["next"] else None
            s["gate"] = None if c["gate"] == "none" else _randn(gen, dt, T, d) if c["gate"] == "full" else _randn(gen, dt, T)
            if c["op"] == "residual":
                s["res"] = _randn(gen, dt, T, d, std=2.0)
            else:
                s["sum"] = _randn(gen, dt, T, d, std=2.0)  # what the forward pass left in out
                s["dout"] = _randn(gen, dt, T, d)
                s["dn"] = _randn(gen, dt, T, d) if c["next"] else None
    if own:
        _plan(s)
    return s


def _prepare_decode(s, gen, dt):
    c = s["case"]
    T, d, E, k, F = c["T"], c["d"], c["E"], c["k"], c["F"]
    std = lambda n: 0.02 if n >= 1024 else 1.0 / math.sqrt(n)  # noqa: E731
    s["x"] = _randn(gen, dt, T, d)
    s["norm"] = _randn(gen, dt, d, std=0.2, mean=1.0) if c["norm"] else None
    s["res"] = _randn(gen, dt, T, d, std=2.0) if c["res"] else None
    s["wr"] = _randn(gen, dt, E, d, std=std(d))
    if c["given"]:  # a routing of the caller's, some slots without an expert (padding)
        ids = torch.rand(T, E, generator=gen, device="cuda").argsort(dim=1)[:, :k].to(torch.int32)
        drop = torch.rand(T, k, generator=gen, device="cuda") < 0.1
        s["ids"] = torch.where(drop, torch.full_like(ids, -1), ids).contiguous()
        s["w"] = torch.softmax(torch.randn(T, k, generator=gen, device="cuda"), dim=1).contiguous()
    for name, n, m in (("wg", F, d), ("wu", F, d), ("wd", d, F)):
        w = _randn(gen, dt, E, n, m, std=std(m))
        if c["weights"] == "e4m3":
            w, s["s" + name[1]] = _e4m3(w)
        s[name] = w


# ---- the framework's calls --------------------------------------------------


def _plan(s):
    """The handles, workspaces and output buffers that a program keeps between calls, and weights in their storage order."""
    import grouped_gemm_gemv_amd as M

    c = s["case"]
    dt = _TYPES[c["dtype"]]
    new = lambda *n, t=dt: torch.zeros(n, dtype=t, device="cuda")  # noqa: E731
    s["M"] = M
    if c["op"] == "dropout":
        s["out"] = {"out": new(c["n"])}
        return
    T, d = c["T"], c["d"]
    if c["op"] == "decode":
        layout = M.LAYOUT_BLOCKED16 if c["blocked"] else M.LAYOUT_ROWS
        s["shape"] = M.Shape(T, d, c["E"], c["k"], c["F"], 0, dt, 0, layout)
        s["ws"] = M.workspace(M.decode_workspace_size(s["shape"]))
        s["out"] = {"out": new(T, d)}
        if c["blocked"]:
            for n in ("wg", "wu", "wd"):
                s[n] = _blocked16(s[n])
        return
    s["shape"] = M.Shape(T, d, 1, 1, 64, dtype=dt)
    s["ws"] = M.workspace(M.residual_workspace_size(s["shape"]))
    if c["op"] == "norm":
        s["out"] = {"n": new(T, d)}
    elif c["op"] == "norm_grad":
        s["out"] = {"dx": new(T, d), "dw": new(d)}
    else:
        gate = {"none": None, "token": (T,), "full": (T, d)}[c["gate"]]
        s["r"] = M.Residual(eps=_EPS, scale=c["scale"], dropout=c["p"])
        if c["op"] == "residual":
            s["out"] = {"out": new(T, d), "n": new(T, d) if c["next"] else None}
        else:
            s["out"] = {"dres": new(T, d), "dy": new(T, d), "dgate": new(*gate) if gate else None,
                        "dpost": new(d) if c["post"] else None, "dnext": new(d) if c["next"] else None}


def _run_own(s):
    M, c, o = s["M"], s["case"], s["out"]
    op = c["op"]
    if op == "dropout":
        M.moe_dropout(s["x"], c["p"], s["rng"], o["out"])
    elif op == "norm":
        M.moe_norm(s["shape"], s["x"], s["w"], o["n"], eps=_EPS)
    elif op == "norm_grad":
        M.moe_norm_backward(s["shape"], s["x"], s["w"], s["dn"], s["dres"], o["dx"], o["dw"], s["ws"], eps=_EPS)
    elif op == "residual":
        M.moe_residual(s["shape"], s["r"], s["res"], s["y"], s["post"], s["gate"], s.get("rng"), s["next"], o["out"],
                       o["n"])
    elif op == "residual_grad":
        M.moe_residual_backward(s["shape"], s["r"], s["sum"], s["y"], s["post"], s["gate"], s.get("rng"), s["next"],
                                s["dout"], s["dn"], o["dres"], o["dy"], o["dgate"], o["dpost"], o["dnext"], s["ws"])
    else:
        wr, ids, w = (None, s["ids"], s["w"]) if c["given"] else (s["wr"], None, None)
        args = (s["shape"], s["x"], s["norm"], wr, None, ids, w, s["wg"], s["wu"], s["wd"])
        if c["weights"] == "e4m3":
            M.moe_decode_fp8(*args, s["sg"], s["su"], s["sd"], s["res"], o["out"], s["ws"], eps=_EPS)
        else:
            M.moe_decode(*args, s["res"], o["out"], s["ws"], eps=_EPS)
    return {name: v for name, v in o.items() if v is not None}


# ---- the plain forms --------------------------------------------------------


def _inv_rms(v):
    return torch.rsqrt((v * v).mean(-1, keepdim=True) + _EPS)


def _drop_scale(rng, p, n):
    """keep_i / (1 - p) of elements 0 .. n - 1, in fp32."""
    t = int(math.floor(float(np.float32(p)) * 65536.0 + 0.5))
    low = 0xFFFFFFFF
    b = torch.arange((n + 7) // 8, device="cuda")
    c0, c1 = b & low, (b >> 32) & low
    c2, c3 = (rng[1] & low).expand_as(b), ((rng[1] >> 32) & low).expand_as(b)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(10):
        m0, m1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # (wraps: the low 64 bits are all that is used)
        c0, c1, c2, c3 = ((m1 >> 32) & low) ^ c1 ^ k0, m1 & low, ((m0 >> 32) & low) ^ c3 ^ k1, m0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], dim=1)
    halves = torch.stack([words & 0xFFFF, words >> 16], dim=2).reshape(-1)[:n]
    return (halves >= t).float() * (65536.0 / (65536 - t))


def _norm_grad(x, w, dn):
    """Gradient of x r(x) w, and of w."""
    r = _inv_rms(x)
    z = dn * w
    return r * z - x * (r * r * r) * (z * x).mean(-1, keepdim=True), (dn * x * r).sum(0)


def _gate(s):
    g = s["gate"].float()
    g = g.unsqueeze(1) if g.dim() == 1 else g
    return 1.0 / (1.0 + torch.exp(-g))


def _keep(s, like):
    c = s["case"]
    return _drop_scale(s["rng"], c["p"], like.numel()).view_as(like) if c["p"] else torch.ones_like(like)


def _run_plain(s):
    c = s["case"]
    op, dt = c["op"], _TYPES[c["dtype"]]
    if op == "dropout":
        return {"out": (s["x"].float() * _drop_scale(s["rng"], c["p"], c["n"])).to(dt)}
    if op == "norm":
        x = s["x"].float()
        return {"n": (x * _inv_rms(x) * s["w"].float()).to(dt)}
    if op == "norm_grad":
        dx, dw = _norm_grad(s["x"].float(), s["w"].float(), s["dn"].float())
        return {"dx": (dx + s["dres"].float()).to(dt), "dw": dw.to(dt)}
    if op == "residual":
        y = s["y"].float()
        v = y * _inv_rms(y) * s["post"].float() if c["post"] else y
        v = v * _keep(s, v) * c["scale"]
        if c["gate"] != "none":
            v = v * _gate(s)
        out = s["res"].float() + v
        outs = {"out": out.to(dt)}
        if c["next"]:
            outs["n"] = (out * _inv_rms(out) * s["next"].float()).to(dt)
        return outs
    if op == "residual_grad":
        outs = {}
        D, y = s["dout"].float(), s["y"].float()
        if c["next"]:
            dx, dw = _norm_grad(s["sum"].float(), s["next"].float(), s["dn"].float())
            D = D + dx
            outs["dnext"] = dw.to(dt)
        outs["dres"] = D.to(dt)
        v = y * _inv_rms(y) * s["post"].float() if c["post"] else y
        D = D * _keep(s, v) * c["scale"]
        if c["gate"] != "none":
            sg = _gate(s)
            dgate = D * v * sg * (1.0 - sg)
            outs["dgate"] = (dgate if c["gate"] == "full" else dgate.sum(1)).to(dt)
            D = D * sg
        if c["post"]:
            D, dw = _norm_grad(y, s["post"].float(), D)
            outs["dpost"] = dw.to(dt)
        outs["dy"] = D.to(dt)
        return outs
    return {"out": _decode(s).to(dt)}


def _decode(s):
    """The block in fp32, over the chosen experts where they are fewer than all, else over all of them."""
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = s["x"].float()
    n = x * _inv_rms(x) * s["norm"].float() if c["norm"] else x
    if c["given"]:
        ids, w = s["ids"].long(), s["w"]
        w = torch.where(ids >= 0, w, torch.zeros_like(w))
        ids = ids.clamp(min=0)
    else:
        top, order = torch.sort(n @ s["wr"].float().t(), dim=1, descending=True, stable=True)
        ids = order[:, :k]
        w = torch.exp(top[:, :k] - top[:, :1])
        w = w / w.sum(1, keepdim=True)

    def matrix(name, at):
        m = s["w" + name][at] if at is not None else s["w" + name]
        if c["weights"] == "e4m3":
            scale = s["s" + name][at] if at is not None else s["s" + name]
            return m.view(torch.float8_e4m3fn).float() * scale.unsqueeze(-1)
        return m.float()

    if T * k < E:
        at, rows, wt = ids.reshape(-1), n.repeat_interleave(k, 0).unsqueeze(1), w.reshape(-1, 1, 1)
    else:
        at, rows = None, n.unsqueeze(0).expand(E, T, -1)
        wt = torch.zeros(T, E, device="cuda").scatter_add_(1, ids, w).t().unsqueeze(-1)
    g = torch.bmm(rows, matrix("g", at).transpose(1, 2))
    u = torch.bmm(rows, matrix("u", at).transpose(1, 2))
    y = torch.bmm(g / (1.0 + torch.exp(-g)) * u, matrix("d", at).transpose(1, 2)) * wt
    y = y.view(T, k, -1).sum(1) if at is not None else y.sum(0)
    return s["res"].float() + y if c["res"] else y


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- 64 bits ----------------------------------------------------------------


def _exact_keep(rng, p, n):
    """The mask over 1 - p in 64 bits, the generator written with 64-bit words of NumPy, a round at a time."""
    t = int(math.floor(float(np.float32(p)) * 65536.0 + 0.5))
    seed, step = (int(v) for v in rng.cpu())
    u = np.uint64
    mask, half = u(0xFFFFFFFF), u(32)
    out = np.empty(n, dtype=np.uint16)
    for at in range(0, n, 1 << 23):  # pieces of 2^20 blocks
        m = min(n - at, 1 << 23)
        block = np.arange(at // 8, (at + m + 7) // 8, dtype=np.uint64)
        ctr = [block & mask, block >> half, np.full_like(block, step & 0xFFFFFFFF), np.full_like(block, step >> 32)]
        key = [seed & 0xFFFFFFFF, seed >> 32]
        for _ in range(10):
            left, right = ctr[0] * u(0xD2511F53), ctr[2] * u(0xCD9E8D57)
            ctr = [(right >> half) ^ ctr[1] ^ u(key[0]), right & mask, (left >> half) ^ ctr[3] ^ u(key[1]), left & mask]
            key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
        out[at:at + m] = np.stack(ctr, axis=1).astype(np.uint32).view(np.uint16).reshape(-1)[:m]
    kept = torch.from_numpy(out.astype(np.int32)).cuda() >= t
    return kept.double() / (1.0 - t / 65536.0)


def exact(case, seed):
    """The outputs from the definitions in 64 bits."""
    c = case
    s = prepare(dict(case, blocked=False) if "blocked" in case else case, seed)
    f = {name: v.double() for name, v in s.items() if torch.is_tensor(v) and v.is_floating_point() and name not in ("wg", "wu", "wd")}
    if c["op"] == "dropout":
        return {"out": f["x"] * _exact_keep(s["rng"], c["p"], c["n"])}
    if c["op"] == "decode":
        return {"out": _exact_decode(s, f)}
    if c["op"] in ("norm", "residual"):
        if c["op"] == "norm":
            return {"n": f["w"] * f["x"] / torch.sqrt(f["x"].square().mean(1, keepdim=True) + _EPS)}
        y = f["y"]
        if c["post"]:
            y = f["post"] * y / torch.sqrt(y.square().mean(1, keepdim=True) + _EPS)
        if c["p"]:
            y = y * _exact_keep(s["rng"], c["p"], y.numel()).view_as(y)
        if c["gate"] != "none":
            y = y * torch.sigmoid(f["gate"].view(c["T"], -1))
        out = f["res"] + c["scale"] * y
        outs = {"out": out}
        if c["next"]:
            outs["n"] = f["next"] * out / torch.sqrt(out.square().mean(1, keepdim=True) + _EPS)
        return outs

    def back(x, w, dn):
        """(d xhat / d x)^T of xhat = x / rms, written with the normalised rows."""
        rms = torch.sqrt(x.square().mean(1, keepdim=True) + _EPS)
        xhat = x / rms
        dhat = dn * w
        return (dhat - xhat * (dhat * xhat).mean(1, keepdim=True)) / rms, torch.einsum("ti,ti->i", dn, xhat)

    if c["op"] == "norm_grad":
        dx, dw = back(f["x"], f["w"], f["dn"])
        return {"dx": dx + f["dres"], "dw": dw}
    outs, dsum, y = {}, f["dout"], f["y"]
    if c["next"]:
        dx, outs["dnext"] = back(f["sum"], f["next"], f["dn"])
        dsum = dsum + dx
    outs["dres"] = dsum
    dv = c["scale"] * dsum
    if c["p"]:
        dv = dv * _exact_keep(s["rng"], c["p"], y.numel()).view_as(y)
    if c["gate"] != "none":
        v = f["post"] * y / torch.sqrt(y.square().mean(1, keepdim=True) + _EPS) if c["post"] else y
        g = f["gate"].view(c["T"], -1)
        slope = torch.sigmoid(g) * torch.sigmoid(-g)
        outs["dgate"] = dv * v * slope if c["gate"] == "full" else (dv * v).sum(1) * slope.view(-1)
        dv = dv * torch.sigmoid(g)
    if c["post"]:
        dv, outs["dpost"] = back(y, f["post"], dv)
    outs["dy"] = dv
    return outs


def _exact_decode(s, f):
    """Expert by expert over the tokens that chose it."""
    c = s["case"]
    x = f["x"]
    if c["norm"]:
        x = f["norm"] * x / torch.sqrt(x.square().mean(1, keepdim=True) + _EPS)
    if c["given"]:
        ids, w = s["ids"].long(), f["w"]
    else:
        z = x @ f["wr"].t()
        ids = torch.argsort(z, dim=1, descending=True, stable=True)[:, :c["k"]]
        w = torch.softmax(torch.gather(z, 1, ids), dim=1)

    def matrix(name, e):
        m = s["w" + name][e]
        if c["weights"] == "e4m3":
            return m.view(torch.float8_e4m3fn).double() * f["s" + name][e].unsqueeze(1)
        return m.double()

    out = f["res"].clone() if c["res"] else torch.zeros_like(x)
    for e in range(c["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        g, u = x[t] @ matrix("g", e).t(), x[t] @ matrix("u", e).t()
        out.index_put_((t,), w[t, j].unsqueeze(1) * ((g * torch.sigmoid(g) * u) @ matrix("d", e).t()), accumulate=True)
    return out
