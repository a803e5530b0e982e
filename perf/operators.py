"""Workloads of the gated linear recurrence, of recurrent steps over a pool of states, and of that
pool's maintenance: what is run, on what inputs, and what each pass has to move.

Six operators, as a user of the package calls them:

  gated_scan_fwd    h_t = a_t h_{t-1} + w_t x_t per channel over whole sequences (prefill)
  gated_scan_bwd    its gradient, measured as the training pass: forward, then backward
  gated_scan_step   the recurrence's single-token form, states in a pool addressed by slot
  decode_step       the delta-rule decode step, states in a pool addressed by slot
  state_copy        pool[dst[i]] = source[src[i]]: forks, reorders, admissions, resets (src -1)
  state_compact     live slots moved into the holes below the live count

with a_t from g_t (gate: log a itself, a logit through the logistic function, or a bounded
log-decay) and w_t = 1 ("plain"), 1 - a_t ("complement") or sqrt(1 - a_t^2) ("norm").

With ``own`` false, run() computes them with elementary torch operations.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
LOWER = -5.0  # lower bound of the log-decay under the "bounded" gate


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # The smallest prefill: one short prompt of a small recurrent layer.
        dict(name="scan_fwd_prompt", op="scan_fwd", B=1, N=1, T=77, D=1024, dtype="bf16",
             g_dtype="bf16", gate="logsigmoid", write="complement", init=False),
        # Long-context prefill of one document (the repository's 131072 tokens), from a carried state.
        dict(name="scan_fwd_document", op="scan_fwd", B=1, N=1, T=131072, D=2048, dtype="bf16",
             g_dtype="f32", gate="log", write="plain", init=True),
        # A training microbatch of 4096-token rows, gates straight from a bf16 projection.
        dict(name="scan_train_rows", op="scan_train", B=8, N=8, T=4096, D=2048, dtype="bf16",
             g_dtype="bf16", gate="logsigmoid", write="norm", init=False),
        # Fine-tuning on packed conversations of ragged lengths in fp32, with carried states.
        dict(name="scan_train_packed", op="scan_train", B=1, N=9, T=20011, D=1288, dtype="f32",
             g_dtype="f32", gate="bounded", write="complement", init=True),
        # Interactive generation: one sequence, one token; the call's latency.
        dict(name="step_single", op="step", N=1, P=8, D=2560, dtype="bf16", g_dtype="bf16",
             gate="logsigmoid", write="norm"),
        # A large serving batch over half of a pool's slots.
        dict(name="step_batch", op="step", N=2048, P=4096, D=4096, dtype="bf16", g_dtype="f32",
             gate="log", write="plain"),
        # Delta-rule decode of a small fp32 model, three requests in a pool of sixteen.
        dict(name="decode_few", op="decode", N=3, P=16, H=4, d=64, dtype="f32", gate="log",
             l2norm=False),
        # Delta-rule decode at the repository's serving size (256 sequences, 32 heads of 128),
        # the states spread over a larger pool.
        dict(name="decode_batch", op="decode", N=256, P=320, H=32, d=128, dtype="bf16",
             gate="logsigmoid", l2norm=True),
        # A prompt's state forked into 7 samples in all layers of a small model.
        dict(name="copy_fork", op="copy", kind="fork", L=12, P=64, H=8, d=64, n=7, width=7),
        # Beam search: 64 requests of 4 beams reordered in place after a step.
        dict(name="copy_beams", op="copy", kind="beams", L=1, P=256, H=16, d=128, n=256, width=4),
        # A small pool of vector states after a handful of requests ended.
        dict(name="compact_few", op="compact", L=4, P=48, H=32, d=1, count=30, holes=5, dk=128),
        # A large pool of matrix states in two layers, a third of it ended.
        dict(name="compact_pool", op="compact", L=2, P=512, H=16, d=128, count=352, holes=96, dk=128),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _channels(rng, hi=8192):
    return 8 * _log(rng, 16, hi // 8)


def draw(rng: random.Random):
    op = rng.choice(["scan_fwd", "scan_train", "step", "decode", "copy", "compact"])
    if op in ("scan_fwd", "scan_train"):
        D = _channels(rng)
        dtype, g_dtype = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        most = (131072 * 2048 if op == "scan_fwd" else 8 * 4096 * 2048) // D // (2 if dtype == "f32" else 1)
        if rng.random() < 0.5:  # rows of one length
            N = B = _log(rng, 1, 64)
            T = _log(rng, 1, max(1, min(131072, most // B)))
        else:                   # packed sequences of ragged lengths
            B, N = 1, _log(rng, 2, 48)
            T = _log(rng, N, max(N, min(131072, most)))
        return dict(op=op, B=B, N=N, T=T, D=D, dtype=dtype, g_dtype=g_dtype,
                    gate=rng.choice(["log", "logsigmoid", "bounded"]),
                    write=rng.choice(["plain", "complement", "norm"]), init=rng.random() < 0.5)
    if op == "step":
        N = _log(rng, 1, 2048)
        D = _channels(rng, 4096)
        dtype, g_dtype = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        return dict(op=op, N=N, P=N + rng.randrange(0, 1 + N), D=D, dtype=dtype, g_dtype=g_dtype,
                    gate=rng.choice(["log", "logsigmoid", "bounded"]),
                    write=rng.choice(["plain", "complement", "norm"]))
    if op == "decode":
        N, d = _log(rng, 1, 256), rng.choice([64, 128])
        return dict(op=op, N=N, P=N + rng.randrange(0, 1 + N // 4), H=rng.choice([1, 3, 4, 8, 16, 32]),
                    d=d, dtype=rng.choice(["bf16", "f32"]), gate=rng.choice(["log", "logsigmoid"]),
                    l2norm=rng.random() < 0.5)
    H, d = rng.choice([1, 2, 5, 8, 16]), rng.choice([64, 128])
    if op == "copy":
        kind, L = rng.choice(["fork", "beams", "admit"]), rng.randint(1, 6)
        most = max(2, 256 * 16 * 128 * 128 // (L * H * d * d))
        if kind == "beams":
            width = rng.randint(2, 8)
            n = width * _log(rng, 1, max(1, min(512, most) // width))
            P = n
        else:
            width = n = _log(rng, 1, min(512, most // 2))
            P = 2 * n + rng.randrange(1, 2 + n)
        return dict(op=op, kind=kind, L=L, P=P, H=H, d=d, n=n, width=width)
    L = rng.randint(1, 4)
    P = _log(rng, 4, max(4, min(2048, 2 * 512 * 16 * 128 * 128 // (L * H * d * d))))
    count = rng.randint(1, P - 1)
    return dict(op=op, L=L, P=P, H=H, d=d, dk=d, count=count,
                holes=rng.randint(0, min(count, P - count)))


# ---------------------------------------------------------------- the inputs

def _gates(gen, shape, gate, dtype):
    """Gate values: log-decays -softplus(n - 3) (half-lives of some ten tokens, long ones among
    them), or logits around 3 (half-lives of a dozen tokens under the logistic function)."""
    n = torch.randn(shape, generator=gen, device=DEVICE)
    if gate == "log":
        z = -torch.nn.functional.softplus(n - 3.0)
    elif gate == "logsigmoid":
        z = n + 3.0
    else:
        z = n - 3.0
    return z.to(dtype)


def _offsets(gen, N, T):
    """N ragged lengths, each at least 1, that sum to T; as offsets, int32."""
    cuts = torch.randperm(T - 1, generator=gen, device=DEVICE)[: N - 1].sort().values + 1
    edge = torch.tensor([0, T], device=DEVICE)
    return torch.cat([edge[:1], cuts, edge[1:]]).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op = case["op"]

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=gen, device=DEVICE) * scale).to(dtype)

    def distinct(n, most):
        return torch.randperm(most, generator=gen, device=DEVICE)[:n].to(torch.int32)

    s = dict(case)
    if op in ("scan_fwd", "scan_train"):
        B, T, D, N = case["B"], case["T"], case["D"], case["N"]
        dt, gdt = DTYPES[case["dtype"]], DTYPES[case["g_dtype"]]
        s["x"] = normal(B, T, D, dtype=dt)
        s["g"] = _gates(gen, (B, T, D), case["gate"], gdt)
        s["init"] = normal(N, D, scale=0.5) if case["init"] else None
        s["cu"] = _offsets(gen, N, T) if N != B else None
        if op == "scan_train":
            s["dout"] = normal(B, T, D, dtype=dt)
            s["dfinal"] = normal(N, D, scale=0.5) if case["init"] else None
    elif op == "step":
        N, P, D = case["N"], case["P"], case["D"]
        s["x"] = normal(N, D, dtype=DTYPES[case["dtype"]])
        s["g"] = _gates(gen, (N, D), case["gate"], DTYPES[case["g_dtype"]])
        s["pool"] = normal(P, D, scale=0.5)
        s["slots"] = distinct(N, P)
    elif op == "decode":
        N, P, H, d, dt = case["N"], case["P"], case["H"], case["d"], DTYPES[case["dtype"]]
        for name in ("q", "k"):
            v = normal(N, H, d)
            s[name] = (v if case["l2norm"] else torch.nn.functional.normalize(v, dim=-1)).to(dt)
        s["v"] = normal(N, H, d, dtype=dt)
        s["g"] = _gates(gen, (N, H, d), case["gate"], torch.float32)
        s["beta"] = torch.sigmoid(normal(N, H))
        s["pool"] = normal(P, H, d, d, scale=0.1)
        s["slots"] = distinct(N, P)
        s["scale"] = d ** -0.5
    elif op == "copy":
        L, P, H, d, n, width = (case[x] for x in ("L", "P", "H", "d", "n", "width"))
        s["pool"] = normal(L, P, H, d, d, scale=0.1)
        s["source"] = None
        if case["kind"] == "beams":  # every beam continues one of its request's beams
            row = torch.arange(n, device=DEVICE)
            pick = torch.randint(0, width, (n,), generator=gen, device=DEVICE)
            s["src"] = (row // width * width + pick).to(torch.int32)
            s["dst"] = row.to(torch.int32)
        elif case["kind"] == "fork":  # one state into n other slots
            some = distinct(n + 1, P)
            s["src"] = some[:1].repeat(n)
            s["dst"] = some[1:].contiguous()
        else:  # prefilled states enter the pool, every fourth slot starts empty
            s["source"] = normal(L, n, H, d, d, scale=0.1)
            row = torch.arange(n, device=DEVICE)
            s["src"] = torch.where(row % 4 == 3, -1, row).to(torch.int32)
            s["dst"] = distinct(n, P)
    else:
        L, P, H, d, dk, count, holes = (case[x] for x in ("L", "P", "H", "d", "dk", "count", "holes"))
        s["pool"] = normal(L, P, H, dk, d, scale=0.1)
        live = torch.zeros(P, dtype=torch.bool, device=DEVICE)
        live[:count] = True
        live[distinct(holes, count).long()] = False
        live[count + distinct(holes, P - count).long()] = True
        s["live"] = live
    return s


# ---------------------------------------------------------------- the calls and the plain forms

def run(s):
    if own:
        return _own(s)
    return {"scan_fwd": _plain_scan, "scan_train": _plain_scan, "step": _plain_step,
            "decode": _plain_decode, "copy": _plain_copy, "compact": _plain_compact}[s["op"]](s)


def _own(s):
    import kimi_delta_attention_17_gb300 as kda
    op = s["op"]
    if op in ("scan_fwd", "scan_train"):
        how = dict(gate=s["gate"], gate_lower=LOWER, write=s["write"])
        train = op == "scan_train"
        out, final, carries = kda.gated_scan_fwd(s["x"], s["g"], s["init"], s["cu"],
                                                 save_carries=train, **how)
        if not train:
            return out, final
        dx, dg, dinit = kda.gated_scan_bwd(s["dout"], s["x"], s["g"], carries, s["cu"],
                                           dfinal_state=s["dfinal"], **how)
        return out, final, dx, dg, dinit
    if op == "step":
        out = kda.gated_scan_step(s["x"], s["g"], s["pool"], slots=s["slots"], gate=s["gate"],
                                  gate_lower=LOWER, write=s["write"])
        return out, s["pool"]
    if op == "decode":
        out = kda.decode_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"], s["pool"],
                              slots=s["slots"], gate=s["gate"], l2norm_qk=s["l2norm"])
        return out, s["pool"]
    if op == "copy":
        kda.state_copy(s["pool"], s["src"], s["dst"], source=s["source"], slot_dim=1)
        return s["pool"]
    new_slot, count = kda.state_compact(s["pool"], s["live"], slot_dim=1)
    return s["pool"], new_slot, count


def _coefficients(g, gate, write):
    """log a, a, 1 - a and w of the gate values, elementwise."""
    if gate == "log":
        la = g
        a, c = torch.exp(la), -torch.expm1(la)
    elif gate == "logsigmoid":
        la = None  # only a and 1 - a are needed
        a, c = 1.0 / (1.0 + torch.exp(-g)), 1.0 / (1.0 + torch.exp(g))
    else:
        la = LOWER / (1.0 + torch.exp(-g))
        a, c = torch.exp(la), -torch.expm1(la)
    if write == "plain":
        w = torch.ones_like(a)
    elif write == "complement":
        w = c
    else:
        w = torch.sqrt(c * (1.0 + a))
    return la, a, c, w


def _bounds(s, device):
    """First and last token of each sequence, over the B * T tokens in a row."""
    B, T = s["B"], s["T"]
    if s["cu"] is None:
        first = torch.arange(B, device=device) * T
        return first, first + T - 1
    cu = s["cu"].long()
    return cu[:-1], cu[1:] - 1


def _doubling(a, b):
    """y_t = a_t y_{t-1} + b_t along the first axis (a_0 unused), by doubling: after k rounds
    (a, b) holds the composition of the 2^k steps that end at t."""
    off, n = 1, a.shape[0]
    while off < n:
        b = torch.cat([b[:off], b[off:] + a[off:] * b[:-off]])
        a = torch.cat([a[:off], a[off:] * a[:-off]])
        off *= 2
    return b


def _plain_scan(s):
    B, T, D = s["B"], s["T"], s["D"]
    x, g = s["x"].float().reshape(-1, D), s["g"].float().reshape(-1, D)
    first, last = _bounds(s, x.device)
    la, a, c, w = _coefficients(g, s["gate"], s["write"])
    init = torch.zeros((s["N"], D), device=x.device) if s["init"] is None else s["init"]
    b = w * x
    b[first] += a[first] * init
    start = a.clone()
    start[first] = 0.0  # nothing crosses from one sequence to the next
    h = _doubling(start, b)
    out, final = h.to(s["x"].dtype).reshape(B, T, D), h[last]
    if s["op"] == "scan_fwd":
        return out, final
    # e_t = dout_t + a_{t+1} e_{t+1}, taken from the last token to the first.
    dout = s["dout"].float().reshape(-1, D).clone()
    if s["dfinal"] is not None:
        dout[last] += s["dfinal"]
    back = torch.zeros_like(a)
    back[:-1] = start[1:]
    e = _doubling(back.flip(0), dout.flip(0)).flip(0)
    before = torch.zeros_like(h)
    before[1:] = h[:-1]
    before[first] = init
    dx = w * e
    dinit = a[first] * e[first]
    # With respect to log a: h depends on it through a h_{t-1} and through w.
    dla = e * a * before
    if s["write"] == "complement":
        dla = dla - e * x * a
    if s["gate"] == "logsigmoid":
        dg = dla * c
        if s["write"] == "norm":  # dw/dg = -a^2 (1 - a) / w = -a^2 w / (1 + a)
            dg = dg - e * x * a * a * w / (1.0 + a)
    else:
        if s["write"] == "norm":
            dla = dla - e * x * a * a / w
        dg = dla if s["gate"] == "log" else dla * la / (1.0 + torch.exp(g))
    return out, final, dx.to(s["x"].dtype).reshape(B, T, D), dg.to(s["g"].dtype).reshape(B, T, D), dinit


def _plain_step(s):
    _, a, _, w = _coefficients(s["g"].float(), s["gate"], s["write"])
    at = s["slots"].long()
    h = a * s["pool"][at] + w * s["x"].float()
    s["pool"][at] = h
    return h.to(s["x"].dtype), s["pool"]


def _plain_decode(s):
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    if s["l2norm"]:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    a = torch.exp(s["g"]) if s["gate"] == "log" else 1.0 / (1.0 + torch.exp(-s["g"]))
    at = s["slots"].long()
    S = s["pool"][at] * a[..., None]
    e = s["beta"][..., None] * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * e[..., None, :]
    o = (S * (s["scale"] * q)[..., None]).sum(-2)
    s["pool"][at] = S
    return o.to(s["v"].dtype), s["pool"]


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    pool = s["pool"]
    source = pool if s["source"] is None else s["source"]
    picked = source[:, src.clamp(min=0)]
    if s["source"] is not None:  # resets occur among admissions only
        picked = torch.where((src < 0).reshape(1, -1, 1, 1, 1), torch.zeros_like(picked[:, :1]), picked)
    pool[:, dst] = picked
    return pool


def _plain_compact(s):
    pool, live = s["pool"], s["live"]
    P = live.shape[0]
    index = torch.arange(P, device=live.device)
    count = live.sum()
    move = live & (index >= count)   # the k-th of these goes into ...
    hole = ~live & (index < count)   # ... the k-th of these
    src, dst = move.nonzero()[:, 0], hole.nonzero()[:, 0]
    new_slot = torch.where(live, index, -1)
    new_slot[src] = dst
    pool[:, dst] = pool[:, src]
    return pool, new_slot.to(torch.int32), count.to(torch.int32).reshape(1)


# ---------------------------------------------------------------- bytes and operations

def work(case):
    op = case["op"]
    if op in ("scan_fwd", "scan_train"):
        n = case["B"] * case["T"] * case["D"]
        x, g, row = BYTES[case["dtype"]], BYTES[case["g_dtype"]], 4 * case["N"] * case["D"]
        state = row * (2 if case["init"] else 1)
        flops = {"plain": 3, "complement": 5, "norm": 7}[case["write"]]
        if op == "scan_fwd":  # x and g in, h and the last states out
            return {"bytes": n * (2 * x + g) + state, "flops": n * flops}
        # x, g and dout in; h, dx and dg out; the states and their gradients. x and g are counted
        # once, although a training step, which has dout only after h, comes back to them.
        return {"bytes": n * (4 * x + 2 * g) + 2 * state, "flops": n * (3 * flops + 4)}
    if op == "step":
        n = case["N"] * case["D"]
        return {"bytes": n * (2 * BYTES[case["dtype"]] + BYTES[case["g_dtype"]] + 8) + 4 * case["N"],
                "flops": n * 5}
    if op == "decode":
        rows, d = case["N"] * case["H"], case["d"]
        return {"bytes": rows * (8 * d * d + 4 * d * BYTES[case["dtype"]] + 4 * d + 4) + 4 * case["N"],
                "flops": rows * d * d * 7}
    slot = 4.0 * case["L"] * case["H"] * case["d"]
    if op == "copy":
        slot *= case["d"]
        n, width = case["n"], case["width"]
        if case["kind"] == "fork":
            moved = 1 + n
        elif case["kind"] == "admit":
            moved = n + (n - n // 4)
        else:
            # A beam that continues itself stays where it is; one that no other beam continues is
            # not read: expected counts for picks spread evenly over the request's beams.
            other = 1.0 - 1.0 / width
            moved = n * other + n * (1.0 - other ** (width - 1))
        return {"bytes": slot * moved + 8 * n, "flops": 0}
    return {"bytes": slot * case["dk"] * 2 * case["holes"] + 5 * case["P"], "flops": 0}


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"scan_fwd": _exact_scan, "scan_train": _exact_scan, "step": _exact_step,
            "decode": _exact_decode, "copy": _exact_copy, "compact": _exact_compact}[case["op"]](s)


def _exact_gate(g, gate):
    """(a, dlog a/dg, log a) in 64 bits."""
    g = g.double()
    if gate == "log":
        la, slope = g, torch.ones_like(g)
    elif gate == "logsigmoid":
        la, slope = torch.nn.functional.logsigmoid(g), torch.sigmoid(-g)
    else:
        la = LOWER * torch.sigmoid(g)
        slope = la * torch.sigmoid(-g)
    return la.exp(), slope, la


def _exact_write(la, write):
    """(w, dw/dlog a) in 64 bits."""
    if write == "plain":
        return torch.ones_like(la), torch.zeros_like(la)
    if write == "complement":
        return -torch.expm1(la), -torch.exp(la)
    w = torch.sqrt(-torch.expm1(2 * la))
    return w, -torch.exp(2 * la) / w


def _exact_scan(s):
    """Token by token, every sequence from its own start; nothing shared with the doubling."""
    D = s["D"]
    if s["cu"] is None:
        spans = [(b * s["T"], (b + 1) * s["T"]) for b in range(s["B"])]
    else:
        cu = s["cu"].tolist()
        spans = list(zip(cu[:-1], cu[1:]))
    x = s["x"].double().reshape(-1, D)
    a, slope, la = _exact_gate(s["g"].reshape(-1, D), s["gate"])
    w, dw = _exact_write(la, s["write"])
    del la
    h = w * x
    N = s["N"]
    init = torch.zeros((N, D), dtype=torch.float64, device=x.device) if s["init"] is None else s["init"].double()
    final = torch.empty_like(init)
    rows = s["cu"] is None  # rows of one length advance together
    groups = [spans] if rows else [[sp] for sp in spans]

    def walk(spans, back, step):
        lo, n = spans[0][0], spans[0][1] - spans[0][0]
        order = range(n - 1, -1, -1) if back else range(n)
        for t in order:
            step(lo + t, slice(lo + t, lo + t + 1 + (len(spans) - 1) * n, n))

    for i, group in enumerate(groups):
        state = [init if rows else init[i:i + 1]]

        def forward(_, at):
            torch.addcmul(h[at], a[at], state[0], out=h[at])
            state[0] = h[at]
        walk(group, False, forward)
        final[(slice(None) if rows else slice(i, i + 1))] = state[0]
    shape = s["x"].shape
    if s["op"] == "scan_fwd":
        return h.reshape(shape), final
    e = s["dout"].double().reshape(-1, D)
    u0 = torch.zeros_like(init) if s["dfinal"] is None else s["dfinal"].double()
    dinit = torch.empty_like(init)
    for i, group in enumerate(groups):
        carry = [u0 if rows else u0[i:i + 1]]

        def backward(_, at):
            e[at] += carry[0]
            carry[0] = a[at] * e[at]
        walk(group, True, backward)
        dinit[(slice(None) if rows else slice(i, i + 1))] = carry[0]
    before = torch.empty_like(h)
    for i, (lo, hi) in enumerate(spans):
        before[lo] = init[i]
        before[lo + 1:hi] = h[lo:hi - 1]
    dla = e * (a * before + x * dw)
    return h.reshape(shape), final, (w * e).reshape(shape), (dla * slope).reshape(shape), dinit


def _exact_step(s):
    a, _, la = _exact_gate(s["g"], s["gate"])
    w, _ = _exact_write(la, s["write"])
    pool = s["pool"].double()
    for_rows = pool.index_select(0, s["slots"].long())
    h = torch.addcmul(w * s["x"].double(), a, for_rows)
    return h, pool.index_copy(0, s["slots"].long(), h)


def _exact_decode(s):
    N, H, d = s["N"], s["H"], s["d"]
    q, k, v = (s[n].double().reshape(N * H, d) for n in ("q", "k", "v"))
    if s["l2norm"]:
        q = q * torch.rsqrt(torch.linalg.vecdot(q, q) + 1e-6)[:, None]
        k = k * torch.rsqrt(torch.linalg.vecdot(k, k) + 1e-6)[:, None]
    a, _, _ = _exact_gate(s["g"].reshape(N * H, d), s["gate"])
    pool = s["pool"].double()
    at = s["slots"].long()
    S = pool[at].reshape(N * H, d, d)
    S.mul_(a[:, :, None])
    seen = torch.bmm(k[:, None, :], S)[:, 0]
    S.baddbmm_(k[:, :, None], (s["beta"].double().reshape(-1, 1) * (v - seen))[:, None, :])
    out = torch.bmm(s["scale"] * q[:, None, :], S)[:, 0]
    pool[at] = S.reshape(N, H, d, d)
    return out.reshape(N, H, d), pool


def _exact_copy(s):
    before = s["pool"] if s["source"] is None else s["source"]
    after = s["pool"].clone()
    for i, j in zip(s["src"].tolist(), s["dst"].tolist()):
        after[:, j] = before[:, i] if i >= 0 else 0.0
    return after.double()


def _exact_compact(s):
    pool, live = s["pool"].clone(), s["live"].tolist()
    n = sum(live)
    to = [i if alive else -1 for i, alive in enumerate(live)]
    holes = iter([i for i in range(n) if not live[i]])
    for i in range(n, len(live)):
        if live[i]:
            to[i] = next(holes)
            pool[:, to[i]] = s["pool"][:, i]
    return pool.double(), None, None
