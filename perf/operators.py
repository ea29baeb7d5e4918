"""The decayed linear attention and the block-norm operators: cases, inputs, plain forms and exact values.

Linear attention with a decay for each value head h (a = exp(g_h), constant over tokens, not trained):

    S_t = a S_{t-1} + k_t v_t^T,      o_t = scale * S_t^T q_t

over whole prompts ("attn_fwd", batched or packed), for one new token of each of N sequences ("attn_step",
the states updated in place), and its gradients ("attn_bwd").  The surroundings of a layer's block
("norm_fwd", "norm_bwd"): y = RMSNorm(b) w_post, r = x + c * sigmoid(u) * y, n = RMSNorm(r) w_pre.

``run`` takes either the plain form (elementary torch operations in fp32, the same algebra regrouped in
chunks so that a long prompt needs no quadratic memory) or, with ``own``, the package's entry points.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6
_CHUNK = 128   # tokens of one block of the plain form


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a short prompt of one user: latency, one ragged chunk
        dict(name="fwd prompt 77", op="attn_fwd", dtype="bf16", lens="77", packed=False, Hqk=16, Hv=32, dk=128, dv=128,
             state=True),
        # the ordinary prefill: 2 x 8192 tokens, query/key heads shared by two value heads
        dict(name="fwd 2x8192", op="attn_fwd", dtype="bf16", lens="8192,8192", packed=False, Hqk=16, Hv=32, dk=128,
             dv=128, state=True),
        # a long context with short requests packed behind it, few heads, odd lengths, one request without tokens
        dict(name="fwd packed 47k", op="attn_fwd", dtype="bf16", lens="40961,0,3007,1,2500,77", packed=True, Hqk=6, Hv=6,
             dk=128, dv=128, state=True),
        # one user decoding: latency
        dict(name="step 1", op="attn_step", dtype="bf16", N=1, pool=1, idle=0, Hqk=16, Hv=32, dk=128, dv=128),
        # a full serving batch, 512 MiB of states
        dict(name="step 256", op="attn_step", dtype="bf16", N=256, pool=256, idle=0, Hqk=16, Hv=32, dk=128, dv=128),
        # a batch with idle rows over a larger pool of states, fp32
        dict(name="step f32 slots", op="attn_step", dtype="f32", N=53, pool=96, idle=11, Hqk=8, Hv=8, dk=64, dv=64),
        # a training step's backward over the ordinary batch
        dict(name="bwd 2x8192", op="attn_bwd", dtype="bf16", lens="8192,8192", packed=False, Hqk=16, Hv=32, dk=128,
             dv=128, state=False),
        # packed training documents of odd lengths, fp32, carried states
        dict(name="bwd f32 packed", op="attn_bwd", dtype="f32", lens="700,0,129,1,514", packed=True, Hqk=4, Hv=8, dk=64,
             dv=64, state=True),
        # one decode batch through a block's surroundings: latency
        dict(name="norm decode 37", op="norm_fwd", dtype="bf16", rows=37, D=2048, gate="full", scaled=True),
        # a prefill's rows
        dict(name="norm 16384", op="norm_fwd", dtype="bf16", rows=16384, D=4096, gate="full", scaled=True),
        # a training step's rows, forward's inputs and both gradients in, six gradients out
        dict(name="norm bwd 16384", op="norm_bwd", dtype="bf16", rows=16384, D=4096, gate="full", scaled=True),
        # a small fp32 model's backward, one gate a token, odd row count and width
        dict(name="norm bwd f32 777", op="norm_bwd", dtype="f32", rows=777, D=1160, gate="row", scaled=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_step", "attn_bwd", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("norm"):
        D = 8 * _log_int(rng, 16, 512)
        return dict(op=op, dtype=dtype, rows=_log_int(rng, 1, 16000 if dtype == "bf16" else 8000),
                    D=D if D != 3072 else 3080, gate=rng.choice(["full", "row", "none"]), scaled=rng.random() < 0.7)
    d = 128 if dtype == "bf16" and rng.random() < 0.7 else rng.choice([32, 64, 128])
    dk, dv = (d, d) if rng.random() < 0.8 else (d, rng.choice([32, 64, 128]))
    Hqk = _log_int(rng, 1, 16)
    Hv = Hqk * rng.choice([1, 1, 2, 3])
    Hv = Hv if Hv <= 32 else Hqk
    if op == "attn_step":
        N = _log_int(rng, 1, 250)
        slots = rng.random() < 0.5
        return dict(op=op, dtype=dtype, N=N, pool=N + (rng.randrange(1, 40) if slots else 0),
                    idle=rng.randrange(0, N // 4 + 1) if slots else 0, Hqk=Hqk, Hv=Hv, dk=dk, dv=dv)
    # tokens x value heads at most those of the largest listed case, fewer in fp32
    most = 2 * 8192 * 32 // (1 if dtype == "bf16" else 8) // Hv
    packed = rng.random() < 0.6
    if packed:
        lens = [rng.choice([0, 1, _log_int(rng, 2, max(3, min(most // 4, 40000)))]) for _ in range(rng.randrange(1, 7))]
        lens.append(_log_int(rng, 2, max(3, min(most // 3, 40000))))
    else:
        B = rng.randrange(1, 5)
        lens = [_log_int(rng, 1, max(2, min(most // B, 20000)))] * B
    return dict(op=op, dtype=dtype, lens=",".join(map(str, lens)), packed=packed, Hqk=Hqk, Hv=Hv, dk=dk, dv=dv,
                state=rng.random() < 0.6)


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
        s.update(x=normal(rows, D), b=normal(rows, D, std=3.0), w_post=normal(D, std=0.1, mean=1.0, dtype=f32),
                 w_pre=normal(D, std=0.1, mean=1.0, dtype=f32),
                 c=normal(D, std=0.1, mean=0.5, dtype=f32) if case["scaled"] else None,
                 u={"full": lambda: normal(rows, D), "row": lambda: normal(rows, 1), "none": lambda: None}[case["gate"]]())
        if case["op"] == "norm_bwd":
            s.update(gr=normal(rows, D), gn=normal(rows, D))
        return s
    Hqk, Hv, dk, dv = case["Hqk"], case["Hv"], case["dk"], case["dv"]
    # slopes from a memory of a few tokens to one of thousands; jittered so that another seed is another model
    steps = torch.linspace(1.0, 11.0, Hv, device="cuda") + 0.5 * torch.rand(Hv, generator=gen, device="cuda")
    s.update(g=-torch.exp2(-steps), scale=dk ** -0.5)

    def projection(*lead):
        """q, k and v as a layer has them: three slices of the rows of one packed projection."""
        p = normal(*lead, 2 * Hqk * dk + Hv * dv)
        q, k, v = p.split([Hqk * dk, Hqk * dk, Hv * dv], dim=-1)
        s.update(q=q.unflatten(-1, (Hqk, dk)), k=k.unflatten(-1, (Hqk, dk)), v=v.unflatten(-1, (Hv, dv)))

    if case["op"] == "attn_step":
        N, pool = case["N"], case["pool"]
        projection(N)
        s["S"] = normal(pool, Hv, dk, dv, std=4.0, dtype=f32)
        s["slots"] = None
        if pool > N or case["idle"]:
            slots = torch.randperm(pool, generator=gen, device="cuda")[:N]
            slots[torch.randperm(N, generator=gen, device="cuda")[:case["idle"]]] = -1   # rows without a request
            s["slots"] = slots.to(torch.int32)
        return s
    lens = _lens(case)
    B, T = (1, sum(lens)) if case["packed"] else (len(lens), lens[0])
    projection(B, T)
    s["lens"], s["cu"] = lens, None
    if case["packed"]:
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    s["S0"] = normal(len(lens), Hv, dk, dv, std=4.0, dtype=f32) if case["state"] else None
    if case["op"] == "attn_bwd":
        s["do"] = normal(B, T, Hv, dv)
        s["dS"] = normal(len(lens), Hv, dk, dv, dtype=f32) if case["state"] else None
    return s


# ------------------------------------------------------------------ the plain forms
def _padded_index(lens, Tp, left, dev):
    """Token positions of every sequence laid out as [sequences, Tp], padded on the left or on the right:
    (index into the flattened tokens, which places hold a token, where each token went)."""
    n = torch.tensor(lens, device=dev)
    start = n.cumsum(0) - n
    pad = Tp - n if left else torch.zeros_like(n)
    pos = torch.arange(Tp, device=dev)[None] - pad[:, None]
    valid = (pos >= 0) & (pos < n[:, None])
    index = torch.where(valid, start[:, None] + pos, 0)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=dev), n)
    back = seq * Tp + torch.arange(int(sum(lens)), device=dev) - start[seq] + pad[seq]
    return index, valid, pos, back


def _scan(q, k, v, g, valid, pos, first, S0):
    """o_t = sum_{j<=t} a^(t-j) (q_t . k_j) v_j + a^(pos_t + first) q_t S0, and sum_j a^(last-j) k_j v_j^T, over
    [sequences, time, heads, features] padded on the left to whole chunks (padded k are zero)."""
    n, T, H, _ = q.shape
    C, nc = _CHUNK, T // _CHUNK
    Q, K, V = (x.reshape(n, nc, C, H, x.shape[-1]).permute(0, 3, 1, 2, 4) for x in (q, k, v))
    i = torch.arange(C, device=q.device, dtype=torch.float32)
    gh = g[:, None, None]
    D = torch.where(i[:, None] >= i, torch.exp(gh * (i[:, None] - i).clamp(min=0)), 0.0)
    o = ((Q @ K.transpose(-1, -2)) * D[:, None]) @ V
    local = (K * torch.exp(gh * (C - 1 - i[:, None]))[:, None]).transpose(-1, -2) @ V
    c = torch.arange(nc, device=q.device, dtype=torch.float32)
    gap = c[:, None] - 1 - c
    M = torch.where(gap >= 0, torch.exp(gh * C * gap.clamp(min=0)), 0.0)
    start = (M @ local.flatten(-2)).reshape(local.shape)
    o = o + (Q * torch.exp(gh * (i[:, None] + 1))[:, None]) @ start
    final = (torch.exp(gh[:, 0] * C * (nc - 1 - c))[..., None, None] * local).sum(2)
    o = o.permute(0, 2, 3, 1, 4).reshape(n, T, H, -1)
    if S0 is not None:
        w = torch.where(valid, 1.0, 0.0)[..., None] * torch.exp((pos.clamp(min=0) + first)[..., None] * g)
        o = o + (q * w[..., None]).transpose(1, 2).matmul(S0).transpose(1, 2)
    return o, final


def _plain_fwd(s, grads):
    q, k, v = (s[x].float().flatten(0, 1) for x in ("q", "k", "v"))
    G = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    g, scale, lens, shape = s["g"], s["scale"], s["lens"], s["v"].shape[:2]
    Tp = max(-(-max(lens) // _CHUNK), 1) * _CHUNK
    n = torch.tensor(lens, device=q.device, dtype=torch.float32)
    whole = torch.exp(n[:, None] * g)[..., None, None]   # a^length
    index, valid, pos, back = _padded_index(lens, Tp, True, q.device)

    def lay(x, index, valid):
        return torch.where(valid[..., None, None], x[index], 0.0)

    def tokens(o, back):
        return o.flatten(0, 1)[back]

    if not grads:
        o, final = _scan(*(lay(x, index, valid) for x in (q, k, v)), g, valid, pos, 1, s["S0"])
        final = final + whole * s["S0"] if s["S0"] is not None else final
        return tokens(o * scale, back).reshape(s["v"].shape).to(s["dtype"]), final
    do = s["do"].float().flatten(0, 1)
    S0t = s["S0"].transpose(-1, -2) if s["S0"] is not None else None
    dq = tokens(_scan(*(lay(x, index, valid) for x in (do, v, k)), g, valid, pos, 1, S0t)[0], back) * scale
    # the other two run backwards in time: padded on the right, then flipped
    index, valid, pos, back = _padded_index(lens, Tp, False, q.device)
    Q, K, V, DO = (lay(x, index, valid).flip(1) for x in (q * scale, k, v, do))
    rvalid, rpos = valid.flip(1), (n.long()[:, None] - 1 - pos).flip(1)
    dSt = s["dS"].transpose(-1, -2) if s["dS"] is not None else None
    dk = tokens(_scan(V, DO, Q, g, rvalid, rpos, 0, dSt)[0].flip(1), back)
    dv, lam = _scan(K, Q, DO, g, rvalid, rpos, 0, s["dS"])
    dv = tokens(dv.flip(1), back)
    dq, dk = (x.unflatten(1, (-1, G)).sum(2).reshape(*shape, -1, x.shape[-1]).to(s["dtype"]) for x in (dq, dk))
    dv = dv.reshape(s["v"].shape).to(s["dtype"])
    if s["S0"] is None:
        return dq, dk, dv
    return dq, dk, dv, lam * torch.exp(g)[:, None, None] + whole * s["dS"]


def _plain_step(s):
    q, k, v = (s[x].float() for x in ("q", "k", "v"))
    G = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    S, slots = s["S"], s["slots"]
    a = torch.exp(s["g"])[:, None, None]
    if slots is None:
        S.mul_(a).add_(k[..., None] * v[..., None, :])
        return (s["scale"] * (q[..., None, :] @ S)[..., 0, :]).to(s["dtype"]), S
    rows = torch.nonzero(slots >= 0)[:, 0]
    at = slots[rows].long()
    new = a * S[at] + k[rows][..., None] * v[rows][..., None, :]
    S[at] = new
    out = torch.zeros_like(v)
    out[rows] = s["scale"] * (q[rows][..., None, :] @ new)[..., 0, :]
    return out.to(s["dtype"]), S


def _plain_norm(s, grads):
    x, b, w_post, w_pre = s["x"].float(), s["b"].float(), s["w_post"], s["w_pre"]
    gate = torch.sigmoid(s["u"].float()) if s["u"] is not None else torch.ones((), device=x.device)
    c = s["c"] if s["c"] is not None else torch.ones((), device=x.device)
    inv_b = torch.rsqrt(b.square().mean(-1, keepdim=True) + _EPS)
    y = b * inv_b * w_post
    r = x + c * gate * y
    inv_r = torch.rsqrt(r.square().mean(-1, keepdim=True) + _EPS)
    if not grads:
        return r.to(s["dtype"]), (r * inv_r * w_pre).to(s["dtype"])
    gr, gn = s["gr"].float(), s["gn"].float()
    rh, bh = r * inv_r, b * inv_b
    h = gn * w_pre
    dr = gr + inv_r * (h - rh * (h * rh).mean(-1, keepdim=True))
    dy = dr * c * gate
    e = dy * w_post
    db = inv_b * (e - bh * (e * bh).mean(-1, keepdim=True))
    out = {"x": dr.to(s["dtype"]), "b": db.to(s["dtype"]), "w_post": (dy * bh).sum(0), "w_pre": (gn * rh).sum(0)}
    if s["c"] is not None:
        out["c"] = (dr * gate * y).sum(0)
    if s["u"] is not None:
        du = dr * c * y * gate * (1 - gate)
        out["u"] = (du.sum(-1, keepdim=True) if s["u"].shape[-1] == 1 else du).to(s["dtype"])
    return out


# ------------------------------------------------------------------ the package's entry points
def _own(s):
    import gated_deltanet_recurrence_03_gb300 as gdn
    op = s["op"]
    if op == "attn_fwd":
        return gdn.gdn_decay_attn_fwd(s["q"], s["k"], s["v"], s["g"], s["S0"], scale=s["scale"], cu_seqlens=s["cu"])
    if op == "attn_step":
        out = gdn.gdn_decay_attn_step(s["q"], s["k"], s["v"], s["g"], s["S"], slots=s["slots"], scale=s["scale"])
        return out, s["S"]
    if op == "attn_bwd":
        grads = gdn.gdn_decay_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["S0"], s["do"], s["dS"], scale=s["scale"],
                                       cu_seqlens=s["cu"], want_grad_S0=s["S0"] is not None)
        return grads if s["S0"] is not None else grads[:3]
    if op == "norm_fwd":
        return gdn.gdn_block_norm_fwd(s["x"], s["b"], s["w_post"], s["w_pre"], gate=s["u"], res_scale=s["c"], eps=_EPS)
    gx, gb, w_post, w_pre, gu, gc = gdn.gdn_block_norm_bwd(s["x"], s["b"], s["w_post"], s["w_pre"], s["gr"], s["gn"],
                                                           gate=s["u"], res_scale=s["c"], eps=_EPS)
    out = {"x": gx, "b": gb, "w_post": w_post, "w_pre": w_pre}
    if gc is not None:
        out["c"] = gc
    if gu is not None:
        out["u"] = gu
    return out


def run(s):
    if own:
        return _own(s)
    if s["op"] == "attn_step":
        return _plain_step(s)
    if s["op"].startswith("norm"):
        return _plain_norm(s, s["op"] == "norm_bwd")
    return _plain_fwd(s, s["op"] == "attn_bwd")


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        rows, D = case["rows"], case["D"]
        u = {"full": D, "row": 1, "none": 0}[case["gate"]]
        vectors = 4 * D * (3 if case["scaled"] else 2)
        if case["op"] == "norm_fwd":
            return {"bytes": rows * (4 * D + u) * e + vectors, "flops": rows * D * 12}
        return {"bytes": rows * (6 * D + 2 * u) * e + 2 * vectors, "flops": rows * D * 40}
    Hqk, Hv, dk, dv = case["Hqk"], case["Hv"], case["dk"], case["dv"]
    state = Hv * dk * dv * 4
    if case["op"] == "attn_step":
        n = case["N"] - case["idle"]
        return {"bytes": 2 * n * state + case["N"] * Hv * dv * e + n * (2 * Hqk * dk + Hv * dv) * e,
                "flops": n * Hv * dk * dv * 5}
    lens = _lens(case)
    t = sum(lens)
    if case["op"] == "attn_fwd":   # q, k, v in, out; the final states, and the initial ones where there are any
        return {"bytes": t * (2 * Hqk * dk + 2 * Hv * dv) * e + len(lens) * state * (2 if case["state"] else 1),
                "flops": t * Hv * dk * dv * 4}
    return {"bytes": t * (4 * Hqk * dk + 3 * Hv * dv) * e + len(lens) * state * (3 if case["state"] else 0),
            "flops": t * Hv * dk * dv * 10}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    def token_loop(s, grads):
        """The token loop, all sequences side by side; one that has ended keeps its state."""
        dev, f64 = s["q"].device, torch.float64
        lens, scale = s["lens"], s["scale"]
        n, Tm = len(lens), max(max(lens), 1)
        G = s["v"].shape[2] // s["q"].shape[2]
        a = torch.exp(s["g"].to(f64))[:, None, None]
        length = torch.tensor(lens, device=dev)
        start = length.cumsum(0) - length

        def rows(x):   # [T, sequences, heads, features], zero past a sequence's end
            flat = torch.cat([x.flatten(0, 1), x.new_zeros(1, *x.shape[2:])])
            t = torch.arange(Tm, device=dev)[:, None]
            return flat[torch.where(t < length, start + t, flat.shape[0] - 1)]

        def at(x, t, rep=1):
            return x[t].to(f64).repeat_interleave(rep, 1)

        q, k, v = rows(s["q"]), rows(s["k"]), rows(s["v"])
        Hv, dk, dv = v.shape[2], q.shape[3], v.shape[3]
        alive = (torch.arange(Tm, device=dev)[:, None] < length)[..., None, None, None]
        S = s["S0"].to(f64) if s["S0"] is not None else torch.zeros(n, Hv, dk, dv, dtype=f64, device=dev)
        one = torch.ones((), dtype=f64, device=dev)
        take = torch.cat([torch.arange(m, device=dev) * n + i for i, m in enumerate(lens)])

        def back(x, heads, d):   # token order again
            return torch.stack(x).flatten(0, 1)[take].reshape(*s["v"].shape[:2], heads, d)

        if not grads:
            out = []
            for t in range(Tm):
                S = torch.where(alive[t], a, one) * S + at(k, t, G)[..., None] * at(v, t)[..., None, :]
                out.append(scale * (at(q, t, G)[..., None, :] @ S)[..., 0, :])
            return back(out, Hv, dv), S
        do = rows(s["do"])
        dq, dkk, dvv = [], [None] * Tm, [None] * Tm
        for t in range(Tm):
            S = torch.where(alive[t], a, one) * S + at(k, t, G)[..., None] * at(v, t)[..., None, :]
            dq.append(scale * (S @ at(do, t)[..., None])[..., 0].unflatten(1, (-1, G)).sum(2))
        lam = s["dS"].to(f64) if s["dS"] is not None else torch.zeros(n, Hv, dk, dv, dtype=f64, device=dev)
        for t in range(Tm - 1, -1, -1):
            lam = lam + scale * at(q, t, G)[..., None] * at(do, t)[..., None, :]
            dkk[t] = (lam @ at(v, t)[..., None])[..., 0].unflatten(1, (-1, G)).sum(2)
            dvv[t] = (at(k, t, G)[..., None, :] @ lam)[..., 0, :]
            lam = torch.where(alive[t], a, one) * lam
        res = back(dq, Hv // G, dk), back(dkk, Hv // G, dk), back(dvv, Hv, dv)
        return res if s["S0"] is None else (*res, lam)

    if case["op"].startswith("attn") and case["op"] != "attn_step":
        lens = _lens(case)
        if max(lens) > 45000 or len(lens) * max(lens) * case["Hv"] * (case["dk"] + case["dv"]) > 2e9:
            return None   # a long loop, or padded fp64 outputs that would not fit beside the rest
    s = prepare(case, seed)
    if case["op"] in ("attn_fwd", "attn_bwd"):
        return token_loop(s, case["op"] == "attn_bwd")
    f64 = torch.float64
    if case["op"] == "attn_step":
        G = s["v"].shape[1] // s["q"].shape[1]
        a = torch.exp(s["g"].to(f64))[None, :, None]
        S, out = s["S"], torch.zeros(*s["v"].shape, dtype=f64, device=s["v"].device)
        S64 = S.to(f64)
        slots = s["slots"].tolist() if s["slots"] is not None else list(range(case["N"]))
        for i, at in enumerate(slots):
            if at < 0:
                continue
            k, q = (s[x][i].to(f64).repeat_interleave(G, 0) for x in ("k", "q"))
            S64[at] = a[0][..., None] * S64[at] + torch.einsum("hk,hv->hkv", k, s["v"][i].to(f64))
            out[i] = case["dk"] ** -0.5 * torch.einsum("hk,hkv->hv", q, S64[at])
        return out, S64
    x, b, wa, wb = (s[n].to(f64) for n in ("x", "b", "w_post", "w_pre"))
    leaves = {"x": x, "b": b, "w_post": wa, "w_pre": wb}
    if s["c"] is not None:
        leaves["c"] = s["c"].to(f64)
    if s["u"] is not None:
        leaves["u"] = s["u"].to(f64)
    for t in leaves.values():
        t.requires_grad_(case["op"] == "norm_bwd")
    y = b / torch.sqrt((b * b).mean(-1, keepdim=True) + _EPS) * wa
    y = y / (1 + torch.exp(-leaves["u"])) if "u" in leaves else y
    r = x + (y * leaves["c"] if "c" in leaves else y)
    n = r / torch.sqrt((r * r).mean(-1, keepdim=True) + _EPS) * wb
    if case["op"] == "norm_fwd":
        return r, n
    loss = (r * s["gr"].to(f64)).sum() + (n * s["gn"].to(f64)).sum()
    return dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
