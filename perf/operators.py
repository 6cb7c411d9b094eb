"""The operators that stand around the block-sparse self-attention of a video DiT block, with
the sizes they are measured at: rotary positions over the (t, y, x) latent grid, applied to Q and
K before it, and cross attention from the latent tokens to an encoder's states of another length,
forward and as a training step (forward and backward).

``listed()`` names fixed cases, ``draw(rng)`` gives more of the same ranges, ``prepare`` makes the
inputs of a case, ``run`` makes one pass (plain torch operations, or the library's kernels where
``own`` is true), ``work`` counts the bytes and operations a pass cannot do without and ``exact``
computes the same outputs in 64 bits.

Rotary: pair p of R/2 (R = dt + dy + dx rotated elements of a head) belongs to the t, y or x axis;
its elements are (2p, 2p + 1) (interleaved) or (p, p + R/2) (half).  The pair turns by
pos_axis * f_p with f_p = theta^(-2i/d_axis), i its index within the axis; scaling changes f_p.
Elements past R and text tokens stay as they are.  The backward is the transpose.

Cross attention: O = softmax(Q K^T / sqrt(D)) V over the valid keys of each batch element, heads
of Q sharing heads of K and V in groups; a row without keys gives O = 0 and lse = -inf.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rope(name, B, T, H, W, heads, D, dims, **more):
    c = dict(op="rope", B=B, T=T, H=H, W=W, n_text=0, heads=heads, heads_k=heads, D=D, dt=dims[0], dy=dims[1],
             dx=dims[2], layout="interleaved", theta=10000.0, scaling="none", factor=1.0, orig_len=0, mscale=1.0,
             dtype="bf16", backward=False, packed=False, origin=0)
    c.update(more)
    if name:
        c["name"] = name
    return c


def _cross(name, B, n_q, n_kv, heads, heads_kv, D, **more):
    c = dict(op="cross", B=B, n_q=n_q, n_kv=n_kv, heads=heads, heads_kv=heads_kv, D=D, dtype="bf16", train=False,
             mask="none", fill=1.0, packed=False)
    c.update(more)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # Q and K of one Wan2.1-1.3B 480p clip, views of a fused QKV projection
        _rope("rope_wan", 1, 21, 30, 52, 12, 128, (44, 42, 42), packed=True),
        # HunyuanVideo 720p with its text tokens, which are not rotated
        _rope("rope_hunyuan_text", 1, 16, 45, 80, 24, 128, (16, 56, 56), n_text=256, theta=256.0),
        # one new token of eight streams far into their sequences, shared K heads: launch latency
        _rope("rope_one_token", 8, 1, 1, 1, 32, 128, (128, 0, 0), heads_k=8, layout="half", theta=500000.0,
              origin=1000000),
        # gradients of Q and K of a clip four times as long as trained on, part of the head, half layout
        _rope("rope_long_backward", 1, 84, 30, 52, 12, 128, (32, 32, 32), layout="half", scaling="yarn", factor=4.0,
              orig_len=21, mscale=0.1 * math.log(4.0) + 1.0, backward=True),
        # the small fp32 grid
        _rope("rope_tiny_f32", 1, 4, 8, 8, 2, 64, (16, 24, 24), dtype="f32"),
        # the latent tokens of one clip over 512 text states, K and V views of a fused projection
        _cross("cross_wan", 1, 32760, 512, 12, 12, 128, packed=True),
        # a long clip over text and image states together (512 + 257), padding inside the list
        _cross("cross_long_masked", 1, 131040, 769, 12, 12, 128, mask="holes", fill=0.8),
        # one learned query per head pooling a clip's latents: the single-token form
        _cross("cross_one_query", 2, 1, 32760, 32, 8, 128, mask="length", fill=0.9),
        # the small fp32 grid over 77 text states
        _cross("cross_tiny_f32", 1, 256, 77, 2, 2, 64, dtype="f32"),
        # a training step of one clip's cross attention
        _cross("cross_wan_train", 1, 32760, 512, 12, 12, 128, train=True),
        # a training step with shared K and V heads and ragged prompts
        _cross("cross_shared_heads_train", 3, 7801, 257, 16, 4, 64, train=True, mask="length", fill=0.6),
        # a training step in fp32: one latent frame
        _cross("cross_frame_train_f32", 1, 1560, 226, 12, 12, 128, dtype="f32", train=True),
    ]


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 0.5 / hi)))))


def draw(rng):
    top = max(work(c)["bytes"] for c in listed()), max(work(c)["flops"] for c in listed())
    if rng.random() < 0.4:
        D = rng.choice((64, 128))
        heads = rng.choice((1, 2, 3, 5, 8, 12, 16, 24, 32, 40))
        left, dims = D // 2, []
        for axis in range(3):
            d = rng.randint(0, left)
            dims.append(2 * d)
            left -= d
        if sum(dims) == 0:
            dims[0] = 2 * rng.randint(1, D // 2)
        rng.shuffle(dims)
        scaling = rng.choice(("none", "none", "linear", "ntk", "yarn"))
        c = _rope(None, rng.randint(1, 4), _log(rng, 1, 84), _log(rng, 1, 60), _log(rng, 1, 90), heads, D, dims,
                  layout=rng.choice(("interleaved", "half")), theta=rng.choice((256.0, 10000.0, 500000.0)),
                  n_text=rng.choice((0, 0, rng.randint(1, 300))), backward=rng.random() < 0.4,
                  packed=rng.random() < 0.4, dtype=rng.choice(("bf16", "bf16", "f32")),
                  origin=rng.choice((0, 0, rng.randint(1, 1000000))), scaling=scaling)
        if not c["packed"]:
            c["heads_k"] = rng.choice([h for h in range(1, heads + 1) if heads % h == 0])
        if scaling != "none":
            c["factor"] = rng.choice((1.5, 2.0, 4.0, 8.0))
            c["orig_len"] = rng.randint(1, 64)
            c["mscale"] = 0.1 * math.log(c["factor"]) + 1.0 if scaling == "yarn" else 1.0
        if work(c)["bytes"] > top[0]:
            c["B"] = 1
        while work(c)["bytes"] > top[0]:
            c["T"] = max(1, c["T"] // 2)
        return c
    few = rng.random() < 0.3      # few queries over many keys, or many queries over an encoder's states
    hkv = rng.choice((1, 2, 3, 4, 8, 12))
    mask = rng.choice(("none", "length", "holes"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    c = _cross(None, rng.randint(1, 4), _log(rng, 1, 300) if few else _log(rng, 64, 131040),
               _log(rng, 64, 32760) if few else _log(rng, 1, 1100), hkv * rng.choice((1, 1, 2, 3, 4, 8)), hkv,
               rng.choice((64, 128)), dtype=dtype, train=rng.random() < 0.5, mask=mask,
               fill=1.0 if mask == "none" else rng.choice((0.3, 0.6, 0.9)), packed=rng.random() < 0.4)
    most = top[1] / (64 if dtype == "f32" else 1)
    if work(c)["flops"] > most:
        c["B"] = 1
    while work(c)["flops"] > most or work(c)["bytes"] > top[0]:
        c["n_q"] = max(1, c["n_q"] * 2 // 3)
        c["n_kv"] = max(1, c["n_kv"] * 5 // 6)
    return c


# ------------------------------------------------------------------ inputs

def _rand(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def prepare(case, seed):
    c, dt = case, _DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    if c["op"] == "rope":
        N = c["T"] * c["H"] * c["W"] + c["n_text"]
        if c["packed"]:
            qkv = _rand(g, (c["B"], N, 3, c["heads"], c["D"]), dt)
            q, k = qkv[:, :, 0], qkv[:, :, 1]
        else:
            q = _rand(g, (c["B"], N, c["heads"], c["D"]), dt)
            k = _rand(g, (c["B"], N, c["heads_k"], c["D"]), dt)
        origin = None
        if c["origin"]:      # how far into its sequence each batch element is
            origin = torch.randint(0, c["origin"] + 1, (c["B"],), generator=g, device="cuda", dtype=torch.int64)
        s = {"case": c, "q": q, "k": k, "origin": origin}
        if own:
            import block_sparse_attention_permute_b200 as bsa
            plan = bsa.Plan(c["B"], c["T"], c["H"], c["W"], 4, 4, 8, c["heads"], c["D"], c["n_text"], dt)
            s["rope"] = plan.rope((c["dt"], c["dy"], c["dx"]), theta=c["theta"], layout=c["layout"],
                                  scaling=c["scaling"], factor=c["factor"], orig_len=c["orig_len"],
                                  mscale=c["mscale"], heads_k=c["heads_k"])
        return s
    B, M, hkv, D = c["B"], c["n_kv"], c["heads_kv"], c["D"]
    # logits of standard deviation 3
    q = _rand(g, (B, c["n_q"], c["heads"], D), dt, 3.0)
    if c["packed"]:
        kv = _rand(g, (B, M, 2, hkv, D), dt)
        k, v = kv[:, :, 0], kv[:, :, 1]
    else:
        k, v = _rand(g, (B, M, hkv, D), dt), _rand(g, (B, M, hkv, D), dt)
    length = mask = None
    u = torch.rand((B, M + 1), generator=g, device="cuda")
    if c["mask"] == "length":
        lo = max(0.0, 2.0 * c["fill"] - 1.0)
        length = ((lo + (1.0 - lo) * u[:, M]) * (M + 1)).to(torch.int32).clamp_(max=M)
    elif c["mask"] == "holes":
        mask = u[:, :M] < c["fill"]
    s = {"case": c, "q": q, "k": k, "v": v, "length": length, "mask": mask}
    if c["train"]:
        s["do"] = _rand(g, (B, c["n_q"], c["heads"], D), dt)
    if own:
        import block_sparse_attention_permute_b200 as bsa
        s["cross"] = bsa.CrossAttention(B, c["n_q"], M, c["heads"], hkv, D, dt)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    if state["case"]["op"] == "rope":
        return _run_rope(state)
    return _run_cross(state)


def _run_rope(s):
    if own:
        f = s["rope"].backward if s["case"]["backward"] else s["rope"].apply
        return f(s["q"], s["k"], t_origin=s["origin"])
    cos, sin = _angles(s["case"], s["origin"])
    if s["case"]["backward"]:
        sin = -sin
    return _turned(s["case"], s["q"], cos, sin), _turned(s["case"], s["k"], cos, sin)


def _axis_frequencies(c, axis, d):
    """Turn per position of each pair of one axis, in 64 bits (d = its elements of the head)."""
    i = torch.arange(0, d, 2, device="cuda", dtype=torch.float64)
    theta, s = c["theta"], c["factor"]
    if c["scaling"] == "ntk" and d > 2:
        theta = theta * s ** (d / (d - 2))
    f = theta ** (-i / max(d, 1))
    if c["scaling"] == "linear":
        f = f / s
    if c["scaling"] == "yarn":      # keep pairs of over 32 turns in the trained length, stretch those under 1
        keep = ((c["orig_len"] * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = (1 - keep) * f / s + keep * f
    return f


def _angles(c, origin):
    """cos and sin of every (batch, video token, pair), the angle formed in 64 bits."""
    T, H, W = c["T"], c["H"], c["W"]
    t, y, x = (torch.arange(n, device="cuda", dtype=torch.float64) for n in (T, H, W))
    t = t[None, :] + (origin.double()[:, None] if origin is not None else 0.0)
    parts = [(t[:, :, None, None, None] * _axis_frequencies(c, 0, c["dt"])).expand(-1, T, H, W, -1),
             (y[None, None, :, None, None] * _axis_frequencies(c, 1, c["dy"])).expand(t.shape[0], T, H, W, -1),
             (x[None, None, None, :, None] * _axis_frequencies(c, 2, c["dx"])).expand(t.shape[0], T, H, W, -1)]
    a = torch.cat(parts, dim=-1).reshape(t.shape[0], T * H * W, 1, -1)
    return (torch.cos(a) * c["mscale"]).float(), (torch.sin(a) * c["mscale"]).float()


def _turned(c, x, cos, sin):
    R, nv = c["dt"] + c["dy"] + c["dx"], c["T"] * c["H"] * c["W"]
    v = x[:, :nv, :, :R].float()
    if c["layout"] == "interleaved":
        a, b = v[..., 0::2], v[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = v[..., : R // 2], v[..., R // 2:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    out = x.clone(memory_format=torch.contiguous_format)
    out[:, :nv, :, :R] = turned.to(x.dtype)
    return out


def _run_cross(s):
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    if own:
        op = s["cross"]
        if not c["train"]:
            return op.forward(q, k, v, kv_len=s["length"], key_mask=s["mask"])
        o, lse = op.forward(q, k, v, kv_len=s["length"], key_mask=s["mask"], return_lse=True)
        dq, dk, dv = op.backward(s["do"], q, k, v, o, lse, kv_len=s["length"], key_mask=s["mask"])
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    G, scale, dt = c["heads"] // c["heads_kv"], c["D"] ** -0.5, q.dtype
    # [B, heads_kv, G * n_q, D]: the heads that share K and V are rows of one product
    qf = _rows(q.float(), G)
    kf, vf = k.float().transpose(1, 2), v.float().transpose(1, 2)
    p = torch.matmul(qf, kf.transpose(2, 3)).mul_(scale)
    hidden = _hidden(s)
    if hidden is not None:
        p.masked_fill_(hidden[:, None, None, :], -math.inf)
    m = p.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p.sub_(m).exp_()
    l = p.sum(dim=-1, keepdim=True)
    p.mul_(torch.where(l > 0, 1.0 / l, torch.zeros_like(l)))
    o = _tokens(torch.matmul(p, vf), G).to(dt)
    if not c["train"]:
        return o
    lse = (m + torch.log(l)).reshape(c["B"], c["heads"], c["n_q"])
    dof = _rows(s["do"].float(), G)
    dv = torch.matmul(p.transpose(2, 3), dof).transpose(1, 2).contiguous()
    dp = torch.matmul(dof, vf.transpose(2, 3))
    ds = dp.sub_((p * dp).sum(dim=-1, keepdim=True)).mul_(p).mul_(scale)
    dq = _tokens(torch.matmul(ds, kf), G)
    dk = torch.matmul(ds.transpose(2, 3), qf).transpose(1, 2).contiguous()
    return {"o": o, "lse": lse, "dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt)}


def _rows(x, G):
    B, N, H, D = x.shape
    return x.transpose(1, 2).reshape(B, H // G, G * N, D)


def _tokens(x, G):
    B, hkv, GN, D = x.shape
    return x.reshape(B, hkv * G, GN // G, D).transpose(1, 2).contiguous()


def _hidden(s):
    """[B, n_kv]: keys that no query sees, or None."""
    if s["length"] is not None:
        return torch.arange(s["case"]["n_kv"], device="cuda")[None, :] >= s["length"][:, None]
    return None if s["mask"] is None else ~s["mask"]


# ------------------------------------------------------------------ work

def work(case):
    c, size = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "rope":
        n = c["B"] * (c["T"] * c["H"] * c["W"] + c["n_text"]) * (c["heads"] + c["heads_k"])
        return {"bytes": 2 * n * c["D"] * size, "flops": 3 * n * (c["dt"] + c["dy"] + c["dx"])}
    nq, nkv = c["B"] * c["n_q"] * c["heads"] * c["D"], c["B"] * c["n_kv"] * c["heads_kv"] * c["D"] * c["fill"]
    pairs = 2 * c["B"] * c["n_q"] * c["heads"] * c["n_kv"] * c["fill"] * c["D"]      # one product
    if not c["train"]:
        return {"bytes": (2 * nq + 2 * nkv) * size, "flops": 2 * pairs}
    # a step: q, do read and o, dq written; k, v read and dk, dv written; lse written; seven products
    return {"bytes": (4 * nq + 4 * nkv) * size + 4 * c["B"] * c["n_q"] * c["heads"], "flops": 7 * pairs}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return _exact_rope(s) if case["op"] == "rope" else _exact_cross(s)


def _exact_rope(s):
    c = s["case"]
    P, nv = [c["dt"] // 2, c["dy"] // 2, c["dx"] // 2], c["T"] * c["H"] * c["W"]
    n = torch.arange(nv, device="cuda")
    grid = [n // (c["H"] * c["W"]), n // c["W"] % c["H"], n % c["W"]]
    out = [x.double().contiguous() for x in (s["q"], s["k"])]
    for b in range(c["B"]):
        turn = torch.empty((nv, sum(P)), device="cuda", dtype=torch.float64)
        p = 0
        for axis in range(3):
            pos = grid[axis].double()
            if axis == 0 and s["origin"] is not None:
                pos = pos + int(s["origin"][b])
            for i in range(P[axis]):
                turn[:, p] = pos * _exact_frequency(c, 2 * P[axis], i)
                p += 1
        if c["backward"]:
            turn = -turn
        z = torch.polar(torch.full_like(turn, c["mscale"]), turn)[:, None, :]
        for o in out:
            v = o[b, :nv, :, : 2 * p]
            if c["layout"] == "interleaved":
                w = torch.view_as_complex(v.reshape(nv, -1, p, 2)) * z
                o[b, :nv, :, : 2 * p] = torch.view_as_real(w).reshape(nv, -1, 2 * p)
            else:
                w = torch.complex(v[..., :p], v[..., p:]) * z
                o[b, :nv, :, : 2 * p] = torch.cat((w.real, w.imag), dim=-1)
    return tuple(out)


def _exact_frequency(c, d, i):
    base = c["theta"]
    if c["scaling"] == "ntk" and d > 2:
        base *= math.pow(c["factor"], d / (d - 2.0))
    f = math.exp(-math.log(base) * 2.0 * i / d)
    if c["scaling"] == "linear":
        return f / c["factor"]
    if c["scaling"] == "yarn":
        turns = c["orig_len"] * f / math.tau
        keep = 0.0 if turns <= 1.0 else 1.0 if turns >= 32.0 else (turns - 1.0) / 31.0
        return f * (keep + (1.0 - keep) / c["factor"])
    return f


def _exact_cross(s):
    c, G = s["case"], s["case"]["heads"] // s["case"]["heads_kv"]
    o = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.full((c["B"], c["heads"], c["n_q"]), -math.inf, device="cuda", dtype=torch.float64)
    dq, dk, dv = (torch.zeros(s[n].shape, device="cuda", dtype=torch.float64) for n in "qkv")
    for b in range(c["B"]):
        seen = torch.arange(c["n_kv"], device="cuda")
        if s["length"] is not None:
            seen = seen[: int(s["length"][b])]
        if s["mask"] is not None:
            seen = seen[s["mask"][b]]
        if seen.numel() == 0:
            continue
        for h in range(c["heads"]):
            x = [s["q"][b, :, h], s["k"][b, seen, h // G], s["v"][b, seen, h // G]]
            x = [t.double().requires_grad_(c["train"]) for t in x]
            logits = x[0] @ x[1].T / math.sqrt(c["D"])
            y = torch.softmax(logits, dim=-1) @ x[2]
            o[b, :, h] = y.detach()
            if c["train"]:
                lse[b, h] = torch.logsumexp(logits.detach(), dim=-1)
                grads = torch.autograd.grad(y, x, s["do"][b, :, h].double())
                dq[b, :, h] = grads[0]
                dk[b, seen, h // G] += grads[1]
                dv[b, seen, h // G] += grads[2]
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if c["train"] else o
