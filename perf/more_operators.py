"""Workloads of what stands around a delta-rule layer: the norm before it and the gradients of both
norms, several tokens a row over a pool of states, and states kept in 8 bits. What is run, on what
inputs, and what each pass has to move.

As a user of the package calls them:

  rmsnorm_quant            h = x + residual; y = w h / rms(h) in e4m3 with scales (a projection's input)
  rmsnorm_fwd, _bwd        the same norm in training: forward, then backward
  output_gate_rmsnorm_bwd  gradient of w o / rms(o) sigmoid(z), per token and head
  state_quantize           slots of a pool of fp32 states into a store of 8-bit codes with scales
  state_dequantize         and back into a pool
  decode_tokens            the delta rule over several tokens a row, states in a pool by slot

The norm takes h as it is stored: rounded to the residual's type where there is one. A store's block of
consecutive values with largest magnitude m has scale m / top and codes round(x * (top / m)), top = 127
with int8 (ties to even) and 448 with e4m3; the factor top / m and the products are fp32 numbers, and a
block with m < 2^-100 is stored as zeros.

With ``own`` false, run() computes them with elementary torch operations.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
STORE = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}
EPS = 1e-6
L2_EPS = 1e-6
SCALE_BLOCK = 128  # values of a row under one scale ("block")
TINY = 2.0 ** -100


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # Interactive generation: the norm before a layer's fp8 projections, one token; the call's latency.
        dict(name="quant_token", op="quant", rows=1, D=2560, dtype="bf16", residual="bf16", block="row"),
        # Prefill of a 131072-token document: residual added, normalised and quantised in one pass.
        dict(name="quant_document", op="quant", rows=131072, D=4096, dtype="bf16", residual="bf16",
             block="block"),
        # A training microbatch of 4096-token rows in bf16 with a bf16 residual stream.
        dict(name="train_rows", op="train", rows=32768, D=2048, dtype="bf16", residual="bf16"),
        # Fine-tuning on packed conversations in fp32, an odd number of tokens and a ragged width.
        dict(name="train_packed", op="train", rows=20011, D=1288, dtype="f32", residual="f32"),
        # The output norm's gradient on one short sequence of a small fp32 model.
        dict(name="gate_grad_prompt", op="gate", tokens=77, H=4, d=64, dtype="f32"),
        # The output norm's gradient on a training microbatch at the repository's 32 heads of 128.
        dict(name="gate_grad_rows", op="gate", tokens=32768, H=32, d=128, dtype="bf16"),
        # One request of a small model parked over 12 layers, and resumed elsewhere.
        dict(name="park_one", op="park", store="int8", L=12, P=64, H=8, d=64, n=1),
        # A serving batch preempted: 256 states of 1 MiB parked, and resumed.
        dict(name="park_batch", op="park", store="int8", L=1, P=320, H=16, d=128, n=256),
        # A cached prefix's state into the slots of 7 samples, over 12 layers.
        dict(name="resume_prefix", op="resume", store="e4m3", L=12, P=64, H=8, d=64, n=7, shared=True),
        # A batch of parked requests back into the pool, two layers.
        dict(name="resume_batch", op="resume", store="e4m3", L=2, P=352, H=16, d=128, n=256, shared=False),
        # Drafts of 4 tokens verified for three requests of a small fp32 model: outputs, no state written.
        dict(name="tokens_verify_few", op="tokens", N=3, P=16, K=4, H=4, d=64, dtype="f32", gate="log",
             l2norm=False, commit=False),
        # Accepted tokens of a serving batch committed (256 sequences, 32 heads of 128, up to 8 tokens each).
        dict(name="tokens_commit_batch", op="tokens", N=256, P=320, K=8, H=32, d=128, dtype="bf16",
             gate="logsigmoid", l2norm=True, commit=True),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["quant", "train", "gate", "park", "resume", "tokens"])
    if op in ("quant", "train"):
        D = 8 * _log(rng, 8, 2048)
        dtype, residual = rng.choice([("bf16", "none"), ("bf16", "bf16"), ("bf16", "f32"),
                                      ("f32", "none"), ("f32", "f32")])
        most = (131072 * 4096 if op == "quant" else 32768 * 2048) // D // (2 if residual == "f32" else 1)
        case = dict(op=op, rows=_log(rng, 1, min(131072, most)), D=D, dtype=dtype, residual=residual)
        return dict(case, block=rng.choice(["row", "block"])) if op == "quant" else case
    if op == "gate":
        H, d, dtype = rng.choice([1, 3, 4, 8, 16, 32]), rng.choice([64, 128]), rng.choice(["bf16", "f32"])
        most = 32768 * 32 * 128 // (H * d) // (2 if dtype == "f32" else 1)
        return dict(op=op, tokens=_log(rng, 1, min(131072, most)), H=H, d=d, dtype=dtype)
    if op == "tokens":
        N, d = _log(rng, 1, 256), rng.choice([64, 128])
        return dict(op=op, N=N, P=N + rng.randrange(0, 1 + N // 4), K=rng.choice([1, 2, 3, 4, 5, 6, 8]),
                    H=rng.choice([1, 3, 4, 8, 16, 32]), d=d, dtype=rng.choice(["bf16", "f32"]),
                    gate=rng.choice(["log", "logsigmoid"]), l2norm=rng.random() < 0.5,
                    commit=rng.random() < 0.5)
    store, L = rng.choice(["int8", "e4m3"]), rng.randint(1, 12)
    H, d = rng.choice([1, 2, 5, 8, 16]), rng.choice([64, 128])
    most = max(1, (256 if op == "park" else 512) * 16 * 128 * 128 // (L * H * d * d))
    n = _log(rng, 1, min(512, most))
    case = dict(op=op, store=store, L=L, P=n + rng.randrange(0, 1 + n // 2), H=H, d=d, n=n)
    return dict(case, shared=rng.random() < 0.25) if op == "resume" else case


# ---------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op = case["op"]

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return torch.randn(shape, generator=gen, device=DEVICE).mul_(scale).to(dtype)

    def distinct(n, most):
        return torch.randperm(most, generator=gen, device=DEVICE)[:n].to(torch.int32)

    s = dict(case)
    if op in ("quant", "train"):
        rows, D, dt = case["rows"], case["D"], DTYPES[case["dtype"]]
        # Layer outputs of order one on a residual stream some times as large, with a few large channels.
        s["x"] = normal(rows, D, dtype=dt)
        s["res"] = None
        if case["residual"] != "none":
            loud = 1.0 + 15.0 * (torch.rand(D, generator=gen, device=DEVICE) < 0.01)
            s["res"] = (normal(rows, D, scale=3.0) * loud).to(DTYPES[case["residual"]])
        s["w"] = 1.0 + normal(D, scale=0.2)
        if op == "train":
            s["dy"] = normal(rows, D, dtype=dt)
            s["dh"] = None if s["res"] is None else normal(rows, D, dtype=s["res"].dtype)
    elif op == "gate":
        shape, dt = (case["tokens"], case["H"], case["d"]), DTYPES[case["dtype"]]
        s["o"], s["z"], s["dout"] = normal(*shape, dtype=dt), normal(*shape, dtype=dt), normal(*shape, dtype=dt)
        s["w"] = 1.0 + normal(case["d"], scale=0.2)
    elif op in ("park", "resume"):
        L, P, H, d, n = (case[x] for x in ("L", "P", "H", "d", "n"))
        kind, top = STORE[case["store"]]
        rows = torch.exp(normal(H, d, 1))  # a state's rows (key channels) differ in size with their decays
        if op == "park":
            s["pool"] = normal(L, P, H, d, d, scale=0.1).mul_(rows)
            s["src"] = distinct(n, P)
            s["at"] = distinct(n, n)  # places in the store
            s["kept"] = torch.zeros((L, n, H, d, d), dtype=kind, device=DEVICE)
            s["scales"] = torch.zeros((L, n, H, d), device=DEVICE)
            s["to"] = torch.arange(n, dtype=torch.int32, device=DEVICE)
            s["back"] = torch.zeros((L, n, H, d, d), device=DEVICE)
        else:
            x = normal(L, n, H, d, d, scale=0.1).mul_(rows)
            most = x.abs().amax(-1, keepdim=True)
            codes = x.mul_(torch.full_like(most, top) / most)
            s["kept"] = (codes.round_() if kind == torch.int8 else codes).to(kind)
            s["scales"] = (most * (1.0 / top)).squeeze(-1)
            s["src"] = distinct(1, n).repeat(n) if case["shared"] else distinct(n, n)
            s["to"] = distinct(n, P)
            s["back"] = normal(L, P, H, d, d, scale=0.1)
    else:
        N, P, K, H, d, dt = case["N"], case["P"], case["K"], case["H"], case["d"], DTYPES[case["dtype"]]
        for name in ("q", "k"):
            v = normal(N, K, H, d)
            s[name] = (v if case["l2norm"] else torch.nn.functional.normalize(v, dim=-1)).to(dt)
        s["v"] = normal(N, K, H, d, dtype=dt)
        z = normal(N, K, H, d)  # half-lives of some ten tokens, long ones among them
        s["g"] = -torch.nn.functional.softplus(z - 3.0) if case["gate"] == "log" else z + 3.0
        s["beta"] = torch.sigmoid(normal(N, K, H))
        s["pool"] = normal(P, H, d, d, scale=0.1)
        s["slots"] = distinct(N, P)
        # Drafts are verified whole; of accepted ones each request has its own number, none among them.
        s["counts"] = torch.randint(0, K + 1, (N,), generator=gen, device=DEVICE).to(torch.int32) \
            if case["commit"] else None
        s["scale"] = d ** -0.5
    return s


# ---------------------------------------------------------------- the calls and the plain forms

def run(s):
    if own:
        return _own(s)
    return {"quant": _plain_quant, "train": _plain_train, "gate": _plain_gate, "park": _plain_park,
            "resume": _plain_resume, "tokens": _plain_tokens}[s["op"]](s)


def _own(s):
    import kimi_delta_attention_17_gb300 as kda
    op = s["op"]
    if op == "quant":
        q, scales, h = kda.rmsnorm_quant(s["x"], s["w"], EPS, residual=s["res"], scale_per=s["block"])
        return q, scales, h if s["res"] is not None else None
    if op == "train":
        y, h, rstd = kda.rmsnorm_fwd(s["x"], s["w"], EPS, residual=s["res"], save_rstd=True)
        dx, dres, dw = kda.rmsnorm_bwd(s["dy"], h, rstd, s["w"], dh=s["dh"])
        if s["res"] is None:
            return y, dx, dw
        return y, h, dx, dres, dw
    if op == "gate":
        return kda.output_gate_rmsnorm_bwd(s["dout"], s["o"], s["z"], s["w"], EPS)
    if op == "park":
        kda.state_quantize(s["pool"], s["src"], s["kept"], s["scales"], s["at"], slot_dim=1)
        kda.state_dequantize(s["kept"], s["scales"], s["at"], s["back"], s["to"], slot_dim=1)
        return s["back"], s["scales"]
    if op == "resume":
        kda.state_dequantize(s["kept"], s["scales"], s["src"], s["back"], s["to"], slot_dim=1)
        return s["back"]
    out = kda.decode_tokens(s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"], s["pool"],
                            slots=s["slots"], counts=s["counts"], write_state=s["commit"],
                            gate=s["gate"], l2norm_qk=s["l2norm"])
    return (out, s["pool"]) if s["commit"] else out


def _plain_sum(s):
    """h as stored, and as fp32."""
    if s["res"] is None:
        return s["x"], s["x"].float()
    h = (s["x"].float() + s["res"].float()).to(s["res"].dtype)
    return h, h.float()


def _plain_quant(s):
    h, f = _plain_sum(s)
    y = s["w"] * (f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS))
    rows, D = y.shape
    size = D if s["block"] == "row" else SCALE_BLOCK
    short = -D % size
    if short:  # the last block of a row is a short one
        y = torch.nn.functional.pad(y, (0, short))
    y = y.reshape(rows, -1, size)
    most = y.abs().amax(-1, keepdim=True)
    q = (y * (torch.full_like(most, 448.0) / most)).to(torch.float8_e4m3fn)
    q = q.reshape(rows, -1)
    q = q[:, :D].contiguous() if short else q
    scales = (most * (1.0 / 448.0)).squeeze(-1)
    return q, scales, h if s["res"] is not None else None


def _plain_train(s):
    h, f = _plain_sum(s)
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    n = f * r
    y = (s["w"] * n).to(s["x"].dtype)
    dy = s["dy"].float()
    u = s["w"] * dy
    d = r * (u - n * (u * n).mean(-1, keepdim=True))
    if s["dh"] is not None:
        d = d + s["dh"].float()
    dw = (dy * n).sum(0)
    dx = d.to(s["x"].dtype)
    if s["res"] is None:
        return y, dx, dw
    return y, h, dx, d.to(s["res"].dtype), dw


def _plain_gate(s):
    o, z, dout = (s[n].float() for n in ("o", "z", "dout"))
    r = torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS)
    n = o * r
    sig = 1.0 / (1.0 + torch.exp(-z))
    dn = dout * sig
    u = dn * s["w"]
    do = r * (u - n * (u * n).mean(-1, keepdim=True))
    dz = u * n * (1.0 / (1.0 + torch.exp(z)))
    dt = s["o"].dtype
    return do.to(dt), dz.to(dt), (dn * n).sum((0, 1))


def _plain_restore(s, rows):
    kept = s["kept"].view(torch.uint8)[:, rows].view(s["kept"].dtype)
    return kept.float() * s["scales"][:, rows][..., None]


def _plain_park(s):
    kind, top = STORE[s["store"]]
    x = s["pool"][:, s["src"].long()]
    most = x.abs().amax(-1, keepdim=True)
    some = most >= TINY
    zero = torch.zeros_like(most)
    codes = x * torch.where(some, torch.full_like(most, top) / most, zero)
    at = s["at"].long()
    s["kept"].view(torch.uint8)[:, at] = (codes.round() if kind == torch.int8 else codes).to(kind).view(torch.uint8)
    s["scales"][:, at] = torch.where(some, most * (1.0 / top), zero).squeeze(-1)
    s["back"][:, s["to"].long()] = _plain_restore(s, at)
    return s["back"], s["scales"]


def _plain_resume(s):
    s["back"][:, s["to"].long()] = _plain_restore(s, s["src"].long())
    return s["back"]


def _plain_tokens(s):
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    if s["l2norm"]:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + L2_EPS)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + L2_EPS)
    q = s["scale"] * q
    a = torch.exp(s["g"]) if s["gate"] == "log" else 1.0 / (1.0 + torch.exp(-s["g"]))
    at = s["slots"].long()
    S = s["pool"][at]
    out = torch.zeros_like(v)
    for t in range(s["K"]):
        new = S * a[:, t, :, :, None]
        e = s["beta"][:, t, :, None] * (v[:, t] - (new * k[:, t, :, :, None]).sum(-2))
        new = new + k[:, t, :, :, None] * e[:, :, None, :]
        o = (new * q[:, t, :, :, None]).sum(-2)
        if s["counts"] is None:
            S, out[:, t] = new, o
        else:  # rows whose tokens have ended keep their states
            going = (s["counts"] > t)[:, None, None]
            S = torch.where(going[..., None], new, S)
            out[:, t] = torch.where(going, o, torch.zeros_like(o))
    out = out.to(s["v"].dtype)
    if not s["commit"]:
        return out
    s["pool"][at] = S
    return out, s["pool"]


# ---------------------------------------------------------------- bytes and operations

def work(case):
    op = case["op"]
    if op in ("quant", "train"):
        n, D = case["rows"] * case["D"], case["D"]
        x, h = BYTES[case["dtype"]], 2 * BYTES.get(case["residual"], 0)  # the residual in, h out
        if op == "quant":
            blocks = 1 if case["block"] == "row" else -(-D // SCALE_BLOCK)
            return {"bytes": n * (x + h + 1) + 4 * case["rows"] * blocks + 4 * D, "flops": n * 8}
        # Forward: x (and the residual) in, y (and h) out; backward: dy (and dh) in, dx (and dres) out.
        return {"bytes": n * (4 * x + 2 * h) + 8 * D, "flops": n * 14}
    if op == "gate":
        n = case["tokens"] * case["H"] * case["d"]
        return {"bytes": 5 * n * BYTES[case["dtype"]] + 8 * case["d"], "flops": n * 18}
    if op in ("park", "resume"):
        values = case["L"] * case["H"] * case["d"] ** 2
        codes = values + 4 * values // case["d"]
        n = case["n"]
        if op == "park":
            return {"bytes": n * (8 * values + codes) + 12 * n, "flops": n * values * 4}
        return {"bytes": 4 * n * values + (1 if case["shared"] else n) * codes + 8 * n, "flops": n * values}
    rows, K, d, b = case["N"] * case["H"], case["K"], case["d"], BYTES[case["dtype"]]
    state, tokens, touched = 4 * d * d, K, 1.0
    if case["commit"]:  # counts spread evenly over 0 .. K
        state, tokens, touched = 2 * state, K / 2, K / (K + 1)
    # Tokens' inputs, the outputs of all K places, and the states of rows with tokens.
    return {"bytes": rows * (state * touched + tokens * (3 * d * b + 4 * d + 4) + K * d * b) + 8 * case["N"],
            "flops": rows * tokens * d * d * 7}


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"quant": _exact_norm, "train": _exact_norm, "gate": _exact_gate, "park": _exact_park,
            "resume": _exact_resume, "tokens": _exact_tokens}[case["op"]](s)


def _exact_norm(s):
    """Rows in groups, so that the largest case's 64-bit values fit beside one another."""
    w, D = s["w"].double(), s["D"]
    parts, dw = [], torch.zeros(D, dtype=torch.float64, device=w.device)
    for lo in range(0, s["rows"], 16384):
        cut = slice(lo, lo + 16384)
        h = s["x"][cut].double()
        if s["res"] is not None:
            h = (h + s["res"][cut].double()).to(s["res"].dtype).double()  # h is what is stored
        rms = torch.linalg.vector_norm(h, dim=1).square().div(D).add(EPS).sqrt()
        y = torch.div(h, rms[:, None]).mul_(w)
        if s["op"] == "quant":
            size = D if s["block"] == "row" else SCALE_BLOCK
            most = torch.stack([piece.abs().max(dim=1).values for piece in y.split(size, dim=1)], dim=1)
            factor = (448.0 / most).repeat_interleave(size, dim=1)[:, :D]
            parts.append(((y * factor).float().to(torch.float8_e4m3fn).float(), most / 448.0,
                          h.to(s["res"].dtype).float() if s["res"] is not None else None))
            continue
        dy = s["dy"][cut].double()
        # d/dh of sum(dy w h / rms): (dy w - y_hat <dy w, y_hat> / D) / rms
        hat = h / rms[:, None]
        wdy = dy * w
        dh = wdy.sub(hat * torch.linalg.vecdot(wdy, hat)[:, None] / D).div_(rms[:, None])
        if s["dh"] is not None:
            dh += s["dh"][cut].double()
        dw += torch.linalg.vecdot(dy, hat, dim=0)
        parts.append((y, dh) if s["res"] is None else (y, h, dh, dh))
    whole = [None if p[0] is None else torch.cat(p) for p in zip(*parts)]
    return tuple(whole) if s["op"] == "quant" else (*whole, dw)


def _exact_gate(s):
    """By automatic differentiation of the forward formula in 64 bits, tokens in groups."""
    w = s["w"].double().requires_grad_()
    parts, dw = [], torch.zeros_like(s["w"], dtype=torch.float64)
    for lo in range(0, s["tokens"], 4096):
        cut = slice(lo, lo + 4096)
        o, z = s["o"][cut].double().requires_grad_(), s["z"][cut].double().requires_grad_()
        y = w * o / (o.square().mean(-1, keepdim=True) + EPS).sqrt() * torch.sigmoid(z)
        do, dz, d = torch.autograd.grad(y, (o, z, w), s["dout"][cut].double())
        parts.append((do, dz))
        dw += d
    return (*(torch.cat(p) for p in zip(*parts)), dw)


def _exact_park(s):
    kind, top = STORE[s["store"]]
    scales, back = s["scales"].double(), s["back"].double()
    for i, (src, at, to) in enumerate(zip(s["src"].tolist(), s["at"].tolist(), s["to"].tolist())):
        x = s["pool"][:, src].double()
        most = x.abs().max(dim=-1).values
        factor = (top / most).float().double()             # the factor and the products are fp32 numbers
        codes = (x * factor[..., None]).float()
        codes = codes.round().double() if kind == torch.int8 else codes.to(kind).double()
        scales[:, at] = most / top
        back[:, to] = codes * (most / top)[..., None]
    return back, scales


def _exact_resume(s):
    back = s["back"].double()
    for src, to in zip(s["src"].tolist(), s["to"].tolist()):
        back[:, to] = torch.einsum("lhij,lhi->lhij", s["kept"][:, src].double(), s["scales"][:, src].double())
    return back


def _exact_tokens(s):
    N, K, H, d = s["N"], s["K"], s["H"], s["d"]

    def heads(x):  # [K, N H, ...]
        return x.double().transpose(0, 1).reshape(K, N * H, *x.shape[3:])
    q, k, v, g, beta = (heads(s[n]) for n in ("q", "k", "v", "g", "beta"))
    if s["l2norm"]:
        q = q * torch.rsqrt(torch.linalg.vecdot(q, q) + L2_EPS)[..., None]
        k = k * torch.rsqrt(torch.linalg.vecdot(k, k) + L2_EPS)[..., None]
    a = g.exp() if s["gate"] == "log" else torch.sigmoid(g)
    pool, at = s["pool"].double(), s["slots"].long()
    S = pool[at].reshape(N * H, d, d)
    counts = torch.full((N,), K, device=S.device) if s["counts"] is None else s["counts"].long()
    out = torch.zeros((K, N * H, d), dtype=torch.float64, device=S.device)
    for t in range(K):
        rows = (counts > t).repeat_interleave(H).nonzero()[:, 0]
        if not rows.numel():
            break
        M = S[rows] * a[t, rows, :, None]
        seen = torch.bmm(k[t, rows, None, :], M)[:, 0]
        M.baddbmm_(k[t, rows, :, None], (beta[t, rows, None] * (v[t, rows] - seen))[:, None, :])
        out[t, rows] = torch.bmm(s["scale"] * q[t, rows, None, :], M)[:, 0]
        S[rows] = M
    out = out.reshape(K, N, H, d).transpose(0, 1)
    if not s["commit"]:
        return out
    pool[at] = S.reshape(N, H, d, d)
    return out, pool
