"""The selective state space scan and the layer norm in front of it: cases, inputs, plain forms and exact values.

The scan, per sequence, channel d of group g(d) and state n, with dt = softplus(delta + dt_bias), A = -exp(A_log):

    h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t,      y_t = (sum_n C_t h_t + skip u_t) silu(z_t)

over whole prompts ("scan_fwd", batched or packed), for one new token of each of N sequences ("scan_step", the
states updated in place), and its gradients ("scan_bwd").  The norm ("norm_fwd", "norm_bwd"): r = x + b,
n = (r - mean r) / sqrt(var r + eps) w + bias.

``run`` takes either the plain form (elementary torch operations in fp32; the scan in blocks of tokens, each
combined by doubling) or, with ``own``, the package's entry points.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-5
_BLOCK = 64   # tokens that the plain scan combines at a time


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a short prompt of one user: latency, a ragged length
        dict(name="fwd prompt 77", op="scan_fwd", dtype="bf16", lens="77", packed=False, D=2048, G=1, N=16, gate=True,
             state=True),
        # the ordinary prefill, 2 x 8192 tokens through a wide layer
        dict(name="fwd 2x8192", op="scan_fwd", dtype="bf16", lens="8192,8192", packed=False, D=4096, G=1, N=16,
             gate=True, state=True),
        # a long context with short requests packed behind it, few channels, odd lengths, one request without tokens
        dict(name="fwd packed 47k", op="scan_fwd", dtype="bf16", lens="40961,0,3007,1,2500,77", packed=True, D=1024,
             G=1, N=16, gate=True, state=True),
        # one user decoding: latency
        dict(name="step 1", op="scan_step", dtype="bf16", rows=1, pool=1, idle=0, D=4096, G=1, N=16, gate=True),
        # a full serving batch
        dict(name="step 256", op="scan_step", dtype="bf16", rows=256, pool=256, idle=0, D=4096, G=1, N=16, gate=True),
        # a batch with idle rows over a larger pool of states, fp32, two groups of larger states, odd width
        dict(name="step f32 slots", op="scan_step", dtype="f32", rows=53, pool=96, idle=11, D=1168, G=2, N=64,
             gate=False),
        # a training step's backward over the ordinary batch
        dict(name="bwd 2x8192", op="scan_bwd", dtype="bf16", lens="8192,8192", packed=False, D=4096, G=1, N=16,
             gate=True, state=False),
        # packed training documents of odd lengths, fp32, carried states
        dict(name="bwd f32 packed", op="scan_bwd", dtype="f32", lens="700,0,129,1,514", packed=True, D=520, G=1, N=16,
             gate=True, state=True),
        # one decode batch through a layer's norm: latency
        dict(name="norm decode 37", op="norm_fwd", dtype="bf16", rows=37, D=2048, residual=True, bias=True),
        # a prefill's rows
        dict(name="norm 16384", op="norm_fwd", dtype="bf16", rows=16384, D=4096, residual=True, bias=True),
        # a training step's rows
        dict(name="norm bwd 16384", op="norm_bwd", dtype="bf16", rows=16384, D=4096, residual=True, bias=True),
        # a small fp32 model's backward, no residual, odd row count and width
        dict(name="norm bwd f32 777", op="norm_bwd", dtype="f32", rows=777, D=1160, residual=False, bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_step", "scan_bwd", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("norm"):
        return dict(op=op, dtype=dtype, rows=_log_int(rng, 1, 16000 if dtype == "bf16" else 8000),
                    D=8 * _log_int(rng, 4, 512), residual=rng.random() < 0.7, bias=rng.random() < 0.7)
    N, G = rng.choice([8, 16, 16, 16, 32, 64]), rng.choice([1, 1, 1, 2, 4])
    D = 8 * G * _log_int(rng, 4, 512 // G)
    base = dict(op=op, dtype=dtype, D=D, G=G, N=N, gate=rng.random() < 0.7)
    if op == "scan_step":
        rows = _log_int(rng, 1, max(1, min(250, 256 * 4096 * 16 // (D * N))))
        slots = rng.random() < 0.5
        return dict(base, rows=rows, pool=rows + (rng.randrange(1, 40) if slots else 0),
                    idle=rng.randrange(0, rows // 4 + 1) if slots else 0)
    # tokens x channels x states at most those of the largest listed case, fewer in fp32
    most = 2 * 8192 * 4096 * 16 // (1 if dtype == "bf16" else 4) // (D * N)
    packed = rng.random() < 0.6
    if packed:
        lens = [rng.choice([0, 1, _log_int(rng, 2, max(3, min(most // 8, 20000)))]) for _ in range(rng.randrange(1, 7))]
        lens.append(_log_int(rng, 2, max(3, min(most // 4, 40000))))
    else:
        B = rng.randrange(1, 5)
        lens = [_log_int(rng, 1, max(2, min(most // B, 20000)))] * B
    return dict(base, lens=",".join(map(str, lens)), packed=packed, state=rng.random() < 0.6)


# ------------------------------------------------------------------ inputs
def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, f32 = _DT[case["dtype"]], torch.float32

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)

    s = {"op": case["op"], "dtype": dt}
    if case["op"].startswith("norm"):
        rows, D = case["rows"], case["D"]
        s.update(x=normal(rows, D, mean=0.3), w=normal(D, std=0.1, mean=1.0, dtype=f32),
                 b=normal(rows, D) if case["residual"] else None,
                 bias=normal(D, std=0.1, dtype=f32) if case["bias"] else None)
        if case["op"] == "norm_bwd":
            s.update(gn=normal(rows, D), gr=normal(rows, D) if case["residual"] else None)
        return s
    D, G, N = case["D"], case["G"], case["N"]
    # the usual start of such a layer: rates 1 .. N, steps of 0.001 to 0.1; jittered so that another seed is another model
    rates = torch.arange(1, N + 1, device="cuda", dtype=f32) * torch.exp(0.1 * torch.randn(D, N, generator=gen, device="cuda"))
    step = torch.exp(math.log(0.001) + math.log(100.0) * torch.rand(D, generator=gen, device="cuda"))
    s.update(A_log=torch.log(rates), dt_bias=step + torch.log(-torch.expm1(-step)), skip=normal(D, std=0.1, mean=1.0, dtype=f32))

    def tokens(*lead):
        """What a layer has in hand: the conv's output, the step's projection, B and C as slices of the rows of one
        projection, and the gate as the second half of the rows of another."""
        rank = -(-D // 128) * 8
        proj = normal(*lead, rank + 2 * G * N)
        xz = normal(*lead, 2 * D) if case["gate"] else None
        u = normal(*lead, D, dtype=f32)
        s.update(u=(u * torch.sigmoid(u)).to(dt), delta=normal(*lead, D, std=0.5),
                 B=proj[..., rank:rank + G * N].unflatten(-1, (G, N)), C=proj[..., rank + G * N:].unflatten(-1, (G, N)),
                 z=xz[..., D:] if case["gate"] else None)

    if case["op"] == "scan_step":
        rows, pool = case["rows"], case["pool"]
        tokens(rows)
        s["h"] = normal(pool, D, N, dtype=f32)
        s["slots"] = None
        if pool > rows or case["idle"]:
            slots = torch.randperm(pool, generator=gen, device="cuda")[:rows]
            slots[torch.randperm(rows, generator=gen, device="cuda")[:case["idle"]]] = -1   # rows without a request
            s["slots"] = slots.to(torch.int32)
        return s
    lens = _lens(case)
    B, T = (1, sum(lens)) if case["packed"] else (len(lens), lens[0])
    tokens(B, T)
    s["lens"], s["cu"] = lens, None
    if case["packed"]:
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    s["h0"] = normal(len(lens), D, N, dtype=f32) if case["state"] else None
    if case["op"] == "scan_bwd":
        s["gy"] = normal(B, T, D)
        s["gh"] = normal(len(lens), D, N, dtype=f32) if case["state"] else None
    return s


# ------------------------------------------------------------------ the plain forms
def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs()))


def _double(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from zero (a and b are overwritten): (h, products of a up to t)."""
    s = 1
    while s < a.shape[1]:
        b[:, s:] = b[:, s:] + a[:, s:] * b[:, :-s]
        a[:, s:] = a[:, s:] * a[:, :-s]
        s *= 2
    return b, a


def _views(s):
    """fp32 tokens split by group, [rows, T, G, D / G] and [rows, T, G, 1, N]; dt and the rates A."""
    G = s["B"].shape[-2]
    x = s["delta"].float() + s["dt_bias"]
    split = lambda t: t.unflatten(-1, (G, -1))   # noqa: E731
    A = -torch.exp(s["A_log"]).unflatten(0, (G, -1))
    return split(s["u"].float()), split(_softplus(x)), A, s["B"].float()[..., None, :], s["C"].float()[..., None, :], x


def _boundaries(s):
    """First and last token of each sequence that has tokens, as (batch row, token, sequence)."""
    if s["cu"] is None:
        rows = [(i, 0, n, i) for i, n in enumerate(s["lens"])]
    else:
        rows, at = [], 0
        for i, n in enumerate(s["lens"]):
            rows.append((0, at, at + n, i))
            at += n
    return [r for r in rows if r[2] > r[1]]


def _plain_scan(s, grads):
    u, dt, A, Bm, Cm, x = _views(s)
    n, T, G, P = u.shape
    N = A.shape[-1]
    seqs = _boundaries(s)
    h0 = s["h0"].unflatten(1, (G, P)) if s["h0"] is not None else None
    starts = {(r, t0): i for r, t0, _, i in seqs}
    ends = {(r, t1 - 1): i for r, _, t1, i in seqs}
    if h0 is not None:
        final = h0.clone()
    else:
        final = torch.zeros(len(s["lens"]), G, P, N, device=u.device)
    f32 = dict(dtype=torch.float32, device=u.device)
    sums = torch.empty(n, T, G, P, **f32)
    hs = torch.empty(n, T, G, P, N, **f32) if grads else None
    carry = torch.zeros(n, G, P, N, **f32)
    for at in range(0, T, _BLOCK):
        c = slice(at, min(at + _BLOCK, T))
        a = torch.exp(dt[:, c, ..., None] * A)
        b = (dt[:, c] * u[:, c])[..., None] * Bm[:, c]
        for (r, t), i in starts.items():
            if c.start <= t < c.stop:
                if h0 is not None:
                    b[r, t - at] += a[r, t - at] * h0[i]
                a[r, t - at] = 0.0
        h, prod = _double(a, b)
        h = h + prod * carry[:, None]
        carry = h[:, -1]
        for (r, t), i in ends.items():
            if c.start <= t < c.stop:
                final[i] = h[r, t - at]
        sums[:, c] = (h * Cm[:, c]).sum(-1)
        if grads:
            hs[:, c] = h
    skip = s["skip"].unflatten(0, (G, P))
    full = sums + skip * u
    z = s["z"].float().unflatten(-1, (G, P)) if s["z"] is not None else None
    if not grads:
        y = full * z * torch.sigmoid(z) if z is not None else full
        return y.flatten(-2).to(s["dtype"]), final.flatten(1, 2)
    gy = s["gy"].float().unflatten(-1, (G, P))
    p, out = gy, {}
    if z is not None:
        sg = torch.sigmoid(z)
        p = gy * z * sg
        out["z"] = (gy * full * sg * (1 + z * (1 - sg))).flatten(-2).to(s["dtype"])
    gh = s["gh"].unflatten(1, (G, P)) if s["gh"] is not None else None
    gu, gdt = torch.empty_like(u), torch.empty_like(u)
    gB, gC = torch.empty_like(Bm), torch.empty_like(Cm)
    gA = torch.zeros_like(A)
    gh0 = gh.clone() if gh is not None else torch.zeros_like(final)
    carry = torch.zeros(n, G, P, N, **f32)   # a_{t+1} lam_{t+1} of the block behind
    for at in range((T - 1) // _BLOCK * _BLOCK, -1, -_BLOCK):
        c = slice(at, min(at + _BLOCK, T))
        L = c.stop - c.start
        a = torch.exp(dt[:, c, ..., None] * A)
        b = p[:, c, ..., None] * Cm[:, c]
        prev = torch.zeros_like(a)
        prev[:, 1:] = hs[:, c.start:c.stop - 1]
        if at:
            prev[:, 0] = hs[:, at - 1]
        up = torch.zeros_like(a)   # a_{t+1}, zero behind a sequence's end
        up[:, :-1] = a[:, 1:]
        b[:, -1] += carry
        for (r, t), i in ends.items():
            if c.start <= t < c.stop:
                up[r, t - at] = 0.0
                if gh is not None:
                    b[r, t - at] += gh[i]
        for (r, t), i in starts.items():
            if c.start <= t < c.stop:
                prev[r, t - at] = h0[i] if h0 is not None else 0.0
        lam = _double(up.flip(1), b.flip(1))[0].flip(1)
        carry = a[:, 0] * lam[:, 0]
        for (r, t), i in starts.items():
            if c.start <= t < c.stop:
                gh0[i] = a[r, t - at] * lam[r, t - at]
                if t == at:
                    carry[r] = 0.0
        q = (lam * Bm[:, c]).sum(-1)
        w = lam * a * prev
        gu[:, c] = dt[:, c] * q + skip * p[:, c]
        gdt[:, c] = u[:, c] * q + (A * w).sum(-1)
        gA += (dt[:, c, ..., None] * w).sum((0, 1))
        gB[:, c] = (lam * (dt[:, c] * u[:, c])[..., None]).sum(-2, keepdim=True)
        gC[:, c] = (hs[:, c] * p[:, c, ..., None]).sum(-2, keepdim=True)
        del a, b, prev, up, lam, q, w, L
    gx = gdt.flatten(-2) * torch.sigmoid(x)
    out.update(u=gu.flatten(-2).to(s["dtype"]), delta=gx.to(s["dtype"]), A_log=(gA * A).flatten(0, 1),
               B=gB[..., 0, :].to(s["dtype"]), C=gC[..., 0, :].to(s["dtype"]), skip=(p * u).sum((0, 1)).flatten(),
               dt_bias=gx.sum((0, 1)))
    if h0 is not None:
        out["h0"] = gh0.flatten(1, 2)
    return out


def _plain_step(s):
    u, dt, A, Bm, Cm, _ = _views(s)
    G, P = u.shape[1:]
    h, slots = s["h"].unflatten(1, (G, P)), s["slots"]
    a, write = torch.exp(dt[..., None] * A), (dt * u)[..., None] * Bm
    rows = torch.nonzero(slots >= 0)[:, 0] if slots is not None else None
    if rows is None:
        h.mul_(a).add_(write)
        new = h
    else:
        at = slots[rows].long()
        new = a[rows] * h[at] + write[rows]
        h[at] = new
        u, Cm = u[rows], Cm[rows]
    y = ((new * Cm).sum(-1) + s["skip"].unflatten(0, (G, P)) * u).flatten(-2)
    if s["z"] is not None:
        z = (s["z"] if rows is None else s["z"][rows]).float()
        y = y * z * torch.sigmoid(z)
    if rows is not None:
        y = torch.zeros(s["u"].shape, device=y.device).index_copy(0, rows, y)
    return y.to(s["dtype"]), s["h"]


def _plain_norm(s, grads):
    r = s["x"].float()
    r = r + s["b"].float() if s["b"] is not None else r
    mean = r.mean(-1, keepdim=True)
    inv = torch.rsqrt((r - mean).square().mean(-1, keepdim=True) + _EPS)
    rh = (r - mean) * inv
    if not grads:
        n = rh * s["w"]
        n = (n + s["bias"] if s["bias"] is not None else n).to(s["dtype"])
        return (n, r.to(s["dtype"])) if s["b"] is not None else n
    gn = s["gn"].float()
    h = gn * s["w"]
    gx = inv * (h - h.mean(-1, keepdim=True) - rh * (h * rh).mean(-1, keepdim=True))
    gx = gx + s["gr"].float() if s["gr"] is not None else gx
    out = {"x": gx.to(s["dtype"]), "w": (gn * rh).sum(0)}
    if s["bias"] is not None:
        out["bias"] = gn.sum(0)
    return out


# ------------------------------------------------------------------ the package's entry points
def _own(s):
    import gated_deltanet_recurrence_03_gb300 as gdn
    op = s["op"]
    if op == "norm_fwd":
        n, r = gdn.gdn_layer_norm_fwd(s["x"], s["w"], s["bias"], residual=s["b"], eps=_EPS)
        return (n, r) if s["b"] is not None else n
    if op == "norm_bwd":
        gx, gw, gb = gdn.gdn_layer_norm_bwd(s["x"], s["w"], s["gn"], residual=s["b"], grad_r=s["gr"], eps=_EPS,
                                            want_grad_bias=s["bias"] is not None)
        return {"x": gx, "w": gw, "bias": gb} if gb is not None else {"x": gx, "w": gw}
    parts = dict(skip=s["skip"], dt_bias=s["dt_bias"], z=s["z"])
    if op == "scan_fwd":
        return gdn.gdn_selective_scan_fwd(s["u"], s["delta"], s["A_log"], s["B"], s["C"], s["h0"], cu_seqlens=s["cu"], **parts)
    if op == "scan_step":
        y = gdn.gdn_selective_scan_step(s["u"], s["delta"], s["A_log"], s["B"], s["C"], s["h"], slots=s["slots"], **parts)
        return y, s["h"]
    g = gdn.gdn_selective_scan_bwd(s["u"], s["delta"], s["A_log"], s["B"], s["C"], s["h0"], s["gy"], s["gh"],
                                   cu_seqlens=s["cu"], want_grad_h0=s["h0"] is not None, **parts)
    names = ("u", "delta", "A_log", "B", "C", "skip", "dt_bias", "z", "h0")
    return {n: t for n, t in zip(names, g) if t is not None}


def run(s):
    if own:
        return _own(s)
    if s["op"] == "scan_step":
        return _plain_step(s)
    if s["op"].startswith("norm"):
        return _plain_norm(s, s["op"] == "norm_bwd")
    return _plain_scan(s, s["op"] == "scan_bwd")


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    D = case["D"]
    if case["op"].startswith("norm"):
        rows, res, bias = case["rows"], case["residual"], case["bias"]
        if case["op"] == "norm_fwd":   # x (b) in, n (r) out
            return {"bytes": rows * D * e * (4 if res else 2) + 4 * D * (2 if bias else 1), "flops": rows * D * 8}
        return {"bytes": rows * D * e * (5 if res else 3) + 4 * D * (3 if bias else 2), "flops": rows * D * 20}
    G, N, gate = case["G"], case["N"], case["gate"]
    weights = 4 * D * (N + 2)
    if case["op"] == "scan_step":
        n = case["rows"] - case["idle"]
        return {"bytes": 2 * n * D * N * 4 + n * ((3 if gate else 2) * D + 2 * G * N) * e + case["rows"] * D * e + weights,
                "flops": n * D * (7 * N + 10)}
    lens = _lens(case)
    t, state = sum(lens), D * N * 4 * len(lens)
    if case["op"] == "scan_fwd":
        return {"bytes": t * ((4 if gate else 3) * D + 2 * G * N) * e + state * (2 if case["state"] else 1) + weights,
                "flops": t * D * (7 * N + 10)}
    return {"bytes": t * ((7 if gate else 5) * D + 4 * G * N) * e + state * (3 if case["state"] else 0) + 2 * weights,
            "flops": t * D * (21 * N + 30)}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    f64 = torch.float64
    if case["op"].startswith("norm"):
        s = prepare(case, seed)
        names = [n for n in ("x", "b", "w", "bias") if s[n] is not None]
        v = {n: s[n].to(f64).requires_grad_(case["op"] == "norm_bwd") for n in names}
        r = v["x"] + v["b"] if "b" in v else v["x"]
        dev = r - r.sum(-1, keepdim=True) / case["D"]
        n = dev / torch.sqrt((dev * dev).sum(-1, keepdim=True) / case["D"] + _EPS) * v["w"]
        n = n + v["bias"] if "bias" in v else n
        if case["op"] == "norm_fwd":
            return (n, r) if "b" in v else n
        loss = (n * s["gn"].to(f64)).sum()
        if s["gr"] is not None:
            loss = loss + (r * s["gr"].to(f64)).sum()
        want = [m for m in names if m != "b"]
        return dict(zip(want, torch.autograd.grad(loss, [v[m] for m in want])))

    D, N = case["D"], case["N"]
    bwd = case["op"] == "scan_bwd"
    if case["op"] != "scan_step":
        lens = _lens(case)
        Tm = max(max(lens), 1)
        if Tm > 45000 or (bwd and len(lens) * Tm * D * N > 2.2e9):
            return None   # a long loop, or states of all tokens that would not fit beside the rest
    s = prepare(case, seed)
    rep = D // case["G"]
    A = -torch.exp(s["A_log"].to(f64))

    def softplus(x):
        return torch.logaddexp(x, torch.zeros_like(x))

    if case["op"] == "scan_step":
        h, y = s["h"].to(f64), torch.zeros(s["u"].shape, dtype=f64, device="cuda")
        for i, at in enumerate(s["slots"].tolist() if s["slots"] is not None else range(case["rows"])):
            if at < 0:
                continue
            u, d = s["u"][i].to(f64), softplus(s["delta"][i].to(f64) + s["dt_bias"])
            B, C = (s[m][i].to(f64).repeat_interleave(rep, 0) for m in ("B", "C"))
            h[at] = torch.exp(d[:, None] * A) * h[at] + (d * u)[:, None] * B
            y[i] = torch.einsum("dn,dn->d", C, h[at]) + s["skip"] * u
            if s["z"] is not None:
                z = s["z"][i].to(f64)
                y[i] *= z / (1 + torch.exp(-z))
        return y, h

    # the token loop, all sequences side by side; one that has ended keeps its state
    n = len(lens)
    length = torch.tensor(lens, device="cuda")
    start = length.cumsum(0) - length
    flat = {m: s[m].flatten(0, 1) for m in ("u", "delta", "B", "C", "z", "gy") if s.get(m) is not None}

    def at(m, t):   # token t of every sequence, the last one again where there is none
        return flat[m][(start + torch.clamp(length - 1, max=t).clamp(min=0)).clamp(max=flat[m].shape[0] - 1)].to(f64)

    def parts(t):
        alive = (t < length)[:, None]
        d = softplus(at("delta", t) + s["dt_bias"]) * alive
        u = at("u", t)
        return alive, u, d, torch.exp(d[..., None] * A), at("B", t).repeat_interleave(rep, 1)

    def put(dst, t, value):
        live = torch.nonzero(t < length)[:, 0]
        dst[start[live] + t] = value[live]

    rows = flat["u"].shape[0]
    h = s["h0"].to(f64) if s["h0"] is not None else torch.zeros(n, D, N, dtype=f64, device="cuda")
    y = torch.zeros(rows, D, dtype=f64, device="cuda")
    kept = torch.empty(Tm, n, D, N, dtype=f64, device="cuda") if bwd else None
    for t in range(Tm):
        _, u, d, a, B = parts(t)
        if bwd:
            kept[t] = h   # the state before token t
        h = a * h + (d * u)[..., None] * B
        put(y, t, (h * at("C", t).repeat_interleave(rep, 1)).sum(-1) + s["skip"] * u)
    z = flat["z"].to(f64) if "z" in flat else None
    shape = s["u"].shape
    if not bwd:
        y = y if z is None else y * z / (1 + torch.exp(-z))
        return y.reshape(shape), h
    out = {m: torch.zeros(rows, D, dtype=f64, device="cuda") for m in ("u", "delta")}
    for m in ("B", "C"):
        out[m] = torch.zeros(rows, case["G"], N, dtype=f64, device="cuda")
    gA, gskip = torch.zeros_like(A), torch.zeros(D, dtype=f64, device="cuda")
    lam = s["gh"].to(f64) if s["gh"] is not None else torch.zeros(n, D, N, dtype=f64, device="cuda")
    fold = lambda x: x.unflatten(1, (case["G"], rep)).sum(2)   # noqa: E731
    for t in range(Tm - 1, -1, -1):
        alive, u, d, a, B = parts(t)
        p = at("gy", t) * alive
        if z is not None:
            zt = at("z", t)
            p = p * zt / (1 + torch.exp(-zt))
        prev = kept[t]
        now = a * prev + (d * u)[..., None] * B
        lam = lam + p[..., None] * at("C", t).repeat_interleave(rep, 1)
        q, w = (lam * B).sum(-1), lam * a * prev * alive[..., None]
        put(out["C"], t, fold(p[..., None] * now))
        put(out["B"], t, fold(lam * (d * u)[..., None]))
        put(out["u"], t, d * q + s["skip"] * p)
        put(out["delta"], t, (u * q + (A * w).sum(-1)) / (1 + torch.exp(-(at("delta", t) + s["dt_bias"]))))
        gA += (w * d[..., None]).sum(0) * A
        gskip += (p * u).sum(0)
        lam = a * lam
    out.update(A_log=gA, skip=gskip, dt_bias=out["delta"].sum(0))
    if z is not None:
        sg = 1 / (1 + torch.exp(-z))
        out["z"] = (flat["gy"].to(f64) * y * sg * (1 + z * (1 - sg))).reshape(shape)
    out["u"], out["delta"] = out["u"].reshape(shape), out["delta"].reshape(shape)
    out["B"], out["C"] = (out[m].reshape(s["B"].shape) for m in ("B", "C"))
    if s["h0"] is not None:
        out["h0"] = lam
    return out
