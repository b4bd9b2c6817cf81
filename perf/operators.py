"""The cases by which the training and serving operators around the SSD are measured.

Three operators in five directions, each as a user's program calls it:
  residual_norm            r = residual + scale * x;  out = r / rms(r) * w         (before a block)
  residual_norm_backward   gradients of x, residual and w
  gated_norm               grouped RMS norm with the SiLU gate, either order       (after the SSD)
  gated_norm_backward      gradients of y, z and w
  prefill_backward         every gradient of the gated linear recurrence that prefill computes

`run` computes the plain form (elementary torch operations in 32 bits, 64 where 32 lose
digits) or, with `own`, makes the library's calls.  `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token of one sequence: the norm ahead of a layer in a decode step
        dict(name="norm_decode_1", op="norm", dir="fwd", rows=1, D=2560, io="bf16", res="f32", scale=1.0),
        # the norm ahead of a 2.7B layer over a whole prefill batch (8 x 4096 tokens)
        dict(name="norm_prefill", op="norm", dir="fwd", rows=32768, D=2560, io="bf16", res="f32", scale=0.5),
        # its gradient in a training step of that batch
        dict(name="norm_train", op="norm", dir="bwd", rows=32768, D=2560, io="bf16", res="f32", scale=0.5),
        # odd row count and odd width in fp32: nothing is 16-byte aligned
        dict(name="norm_train_odd_f32", op="norm", dir="bwd", rows=1111, D=777, io="f32", res="f32", scale=1.0),
        # 32 sequences decoding: the gate is a slice of the input projection's row
        dict(name="gate_decode_32", op="gate", dir="fwd", rows=32, D=5120, groups=1, io="bf16", order="gate_first", pad=5456),
        # the gated norm over a prefill batch, 8 norm groups
        dict(name="gate_prefill", op="gate", dir="fwd", rows=16384, D=5120, groups=8, io="bf16", order="gate_first", pad=5456),
        # its gradient in training
        dict(name="gate_train", op="gate", dir="bwd", rows=16384, D=5120, groups=1, io="bf16", order="gate_first", pad=5456),
        # fp32, the norm ahead of the gate, a ragged batch
        dict(name="gate_train_f32", op="gate", dir="bwd", rows=2049, D=1536, groups=1, io="f32", order="norm_first", pad=0),
        # the tiny fp32 SSD core
        dict(name="ssd_tiny_f32", op="ssd", b=1, T=512, H=4, N=64, G=1, io="f32", h0=False, dhf=False, raw=False),
        # ragged sequences, four groups, raw steps, states passed in and out of the sequence
        dict(name="ssd_ragged", op="ssd", b=3, T=1021, H=16, N=128, G=4, io="bf16", h0=True, dhf=True, raw=True),
        # a 130M-shaped layer, one sequence
        dict(name="ssd_130m", op="ssd", b=1, T=4096, H=24, N=128, G=1, io="bf16", h0=False, dhf=False, raw=False),
        # a 2.7B-shaped layer, the training batch
        dict(name="ssd_2p7b", op="ssd", b=8, T=4096, H=80, N=128, G=1, io="bf16", h0=True, dhf=False, raw=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gate", "ssd", "ssd"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "ssd":
        G = rng.choice([1, 1, 2, 4, 8])
        H = G * rng.randint(1, 80 // G)
        N = rng.choice([64, 128, 128])
        b = _log_int(rng, 1, 8)
        T = _log_int(rng, 1, 4096)
        # the fp32 and N = 64 forms do their sums on the fp32 pipes: smaller batches
        most = 2621440 if io == "bf16" and N == 128 else 400000
        while b * T * H > most:
            b, T = (b // 2, T) if b > 1 else (1, T // 2)
        return dict(op="ssd", b=b, T=T, H=H, N=N, G=G, io=io, h0=rng.random() < 0.5, dhf=rng.random() < 0.5,
                    raw=rng.random() < 0.3)
    D = _log_int(rng, 64, 10240)
    if rng.random() < 0.6:
        D = max(64, D // 64 * 64)
    most = 80_000_000
    rows = _log_int(rng, 1, max(1, min(65536, most // D)))
    direction = rng.choice(["fwd", "bwd"])
    if op == "norm":
        return dict(op="norm", dir=direction, rows=rows, D=D, io=io, res=rng.choice(["f32", io]),
                    scale=rng.choice([1.0, 0.5, 0.22]))
    groups = rng.choice([g for g in (1, 2, 4, 8) if D % g == 0])
    return dict(op="gate", dir=direction, rows=rows, D=D, groups=groups, io=io,
                order=rng.choice(["gate_first", "norm_first"]), pad=rng.choice([0, 0, 336, 8 * rng.randint(1, 600)]))


# ---------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    io = _DT[case["io"]]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    st = dict(case=case)
    if case["op"] == "norm":
        rows, D = case["rows"], case["D"]
        st["weight"] = 1.0 + 0.1 * normal(D)
        if case["dir"] == "fwd":
            st["x"] = normal(rows, D, dtype=io)
            st["residual"] = normal(rows, D, std=2.0, dtype=_DT[case["res"]])
        else:
            st["r"] = normal(rows, D, std=2.0, dtype=_DT[case["res"]])
            st["dout"] = normal(rows, D, dtype=io)
            st["dr_out"] = normal(rows, D, dtype=_DT[case["res"]])
    elif case["op"] == "gate":
        rows, D = case["rows"], case["D"]
        st["weight"] = 1.0 + 0.1 * normal(D)
        st["y"] = normal(rows, D, dtype=io)
        st["z"] = normal(rows, D + case["pad"], dtype=io)[:, :D]  # a slice of a wider row
        if case["dir"] == "bwd":
            st["dout"] = normal(rows, D, dtype=io)
    else:
        b, T, H, N, G, P = case["b"], case["T"], case["H"], case["N"], case["G"], 64
        lo, hi = math.log(1e-3), math.log(1e-1)
        u = torch.rand(2, H, generator=g, device="cuda", dtype=torch.float64)
        st["A"] = -torch.exp(u[0] * math.log(16.0)).float()
        bias = torch.log(torch.expm1(torch.exp(lo + (hi - lo) * u[1]))).float()
        z = 0.5 * normal(b, T, H)
        if case["raw"]:
            st["dt"], st["dt_bias"] = z, bias
        else:
            st["dt"], st["dt_bias"] = torch.log1p(torch.exp(z + bias)), None
        st["x"] = normal(b, T, H, P, dtype=io)
        st["B"] = normal(b, T, G, N, dtype=io)
        st["C"] = normal(b, T, G, N, dtype=io)
        st["D"] = 1.0 + 0.1 * normal(H)
        st["h0"] = normal(b, H, P, N, std=0.1) if case["h0"] else None
        st["dy"] = normal(b, T, H, P, dtype=io)
        st["dh_final"] = normal(b, H, P, N, std=0.1) if case["dhf"] else None
    return st


def _eps(case):
    return 1e-5


# ---------------------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        import state_space_model_04_b200 as ssd

        return _own(ssd, case, state)
    if case["op"] == "norm":
        return _plain_norm(case, state)
    if case["op"] == "gate":
        return _plain_gate(case, state)
    return _plain_ssd(case, state)


def _own(ssd, case, s):
    if case["op"] == "norm":
        if case["dir"] == "fwd":
            out, r = ssd.residual_norm(s["x"], s["weight"], s["residual"], scale=case["scale"], eps=_eps(case))
            return dict(out=out, r=r)
        dx, dres, dw = ssd.residual_norm_backward(s["dout"], s["r"], s["weight"], s["dr_out"], scale=case["scale"],
                                                  eps=_eps(case))
        return dict(dx=dx, dres=dres, dw=dw)
    if case["op"] == "gate":
        first = case["order"] == "norm_first"
        if case["dir"] == "fwd":
            return dict(out=ssd.gated_norm(s["y"], s["z"], s["weight"], groups=case["groups"], eps=_eps(case),
                                           norm_before_gate=first))
        dy, dz, dw = ssd.gated_norm_backward(s["dout"], s["y"], s["z"], s["weight"], groups=case["groups"],
                                             eps=_eps(case), norm_before_gate=first)
        return dict(dy=dy, dz=dz, dw=dw)
    g = ssd.prefill_backward(s["dy"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], h0=s["h0"],
                             dh_final=s["dh_final"], dt_raw=case["raw"], dt_bias=s["dt_bias"])
    out = dict(dx=g.dx, ddt=g.ddt, dA=g.dA, dB=g.dB, dC=g.dC, dD=g.dD, dh0=g.dh0)
    if case["raw"]:
        out["ddt_bias"] = g.ddt_bias
    return out


# ---------------------------------------------------------------------------- plain forms
def _plain_norm(case, s):
    w, eps, scale = s["weight"], _eps(case), case["scale"]
    if case["dir"] == "fwd":
        r = s["residual"].float() + scale * s["x"].float()
        out = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + eps) * w
        return dict(out=out.to(s["x"].dtype), r=r.to(s["residual"].dtype))
    r, dout = s["r"].float(), s["dout"].float()
    k = torch.rsqrt((r * r).mean(-1, keepdim=True) + eps)
    n = r * k
    g = dout * w
    dr = k * (g - n * (g * n).mean(-1, keepdim=True)) + s["dr_out"].float()
    return dict(dx=(scale * dr).to(s["dout"].dtype), dres=dr.to(s["r"].dtype), dw=(dout * n).sum(0))


def _plain_gate(case, s):
    rows, D, n, eps = case["rows"], case["D"], case["groups"], _eps(case)
    first = case["order"] == "norm_first"
    y, z = s["y"].float(), s["z"].float()
    w = s["weight"]
    sig = 1.0 / (1.0 + torch.exp(-z))
    gate = z * sig
    v = (y if first else y * gate).view(rows, n, D // n)
    k = torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)
    u = (v * k).view(rows, D)
    if case["dir"] == "fwd":
        return dict(out=(u * w * (gate if first else 1.0)).to(s["y"].dtype))
    dout = s["dout"].float()
    t = dout * gate if first else dout
    dw = (t * u).sum(0)
    gv, uv = (t * w).view(rows, n, D // n), u.view(rows, n, D // n)
    dv = (k * (gv - uv * (gv * uv).mean(-1, keepdim=True))).view(rows, D)
    dgate = dout * u * w if first else dv * y
    dy = dv if first else dv * gate
    dz = dgate * sig * (1.0 + z * (1.0 - sig))
    return dict(dy=dy.to(s["y"].dtype), dz=dz.to(s["y"].dtype), dw=dw)


def _plain_ssd(case, s, Q=64):
    """The chunked dual form's gradients.  With a_t = dt_t A, cs its prefix sum in a chunk,
    L_ij = exp(cs_i - cs_j) for i >= j, S = C B^T, Gm = dy x^T:
      dx_j = dt_j (sum_i S_ij L_ij dy_i + exp(cs_Q - cs_j) dh B_j) + D dy_j   (dh: adjoint of the state leaving)
      dC_i = sum_j Gm_ij L_ij dt_j B_j + exp(cs_i) h^T dy_i                   (h: the state entering)
      dB_j = sum_i Gm_ij L_ij dt_j C_i + dt_j exp(cs_Q - cs_j) dh^T x_j
      da_t = exp(cs_Q) <h, dh> + sum_{i >= t} E_i + sum_{j < t} F_j + sum_{i >= t > j} W_ij
    with W = Gm S L dt, E_i = exp(cs_i) dy_i . h C_i and F_j = dt_j exp(cs_Q - cs_j) x_j . dh B_j."""
    b, T, H, N, G, P = case["b"], case["T"], case["H"], case["N"], case["G"], 64
    hg, nc = H // G, -(-T // Q)
    pad = nc * Q - T
    A, io = s["A"], s["x"].dtype

    def chunks(t, *tail):  # [b,T,...] -> [b,nc,Q,...] in fp32, zero rows at the end
        t = torch.nn.functional.pad(t.float(), (0, 0) * (t.dim() - 2) + (0, pad))
        return t.view(b, nc, Q, *tail)

    if case["raw"]:
        zr = s["dt"] + s["dt_bias"]
        dt = torch.where(zr > 20, zr, torch.log1p(torch.exp(zr)))
    else:
        dt = s["dt"]
    x, dy = chunks(s["x"], G, hg, P), chunks(s["dy"], G, hg, P)
    B, C = chunks(s["B"], G, N), chunks(s["C"], G, N)
    dtc = chunks(dt, H).permute(0, 1, 3, 2)  # [b,nc,H,Q]
    cs = (dtc.double() * A.double()[:, None]).cumsum(-1)
    tot = cs[..., -1]  # [b,nc,H]
    low = torch.ones(Q, Q, device=A.device, dtype=torch.bool).tril()
    L = torch.exp((cs[..., :, None] - cs[..., None, :]).masked_fill(~low, -math.inf).float())  # [b,nc,H,i,j]
    e = torch.exp(cs).float()
    w = torch.exp(tot[..., None] - cs).float()

    def byg(t):
        return t.view(b, nc, G, hg, *t.shape[3:])

    xh, dyh = x.permute(0, 1, 3, 4, 2, 5), dy.permute(0, 1, 3, 4, 2, 5)  # [b,nc,G,hg,Q,P]
    Bg, Cg = B.permute(0, 1, 3, 2, 4)[:, :, :, None], C.permute(0, 1, 3, 2, 4)[:, :, :, None]  # [b,nc,G,1,Q,N]
    wdt = byg(w * dtc)[..., None]
    # the states between chunks: h[c] = sum over earlier chunks of their local states, decayed
    s_loc = (xh * wdt).transpose(-1, -2) @ Bg  # [b,nc,G,hg,P,N]
    g_loc = (dyh * byg(e)[..., None]).transpose(-1, -2) @ Cg
    run_ = torch.cumsum(tot, 1)  # [b,nc,H]: the decay up to the end of chunk c
    before = (run_ - tot).transpose(1, 2)  # up to its start
    after = run_.transpose(1, 2)
    early = torch.ones(nc, nc, device=A.device, dtype=torch.bool).tril(-1)
    pass_ = torch.exp((before[:, :, :, None] - after[:, :, None, :]).masked_fill(~early, -math.inf)).float()  # [b,H,c,c']
    flat = lambda t: t.reshape(b, nc, H, P * N).transpose(1, 2)  # noqa: E731
    h = pass_ @ flat(s_loc)  # [b,H,nc,PN]
    dh = pass_.transpose(-1, -2) @ flat(g_loc)
    if s["h0"] is not None:
        h = h + torch.exp(before).float()[..., None] * s["h0"].view(b, H, 1, P * N)
    left = (after[:, :, -1:] - after)  # the decay behind chunk c
    if s["dh_final"] is not None:
        dh = dh + torch.exp(left).float()[..., None] * s["dh_final"].view(b, H, 1, P * N)
    back = lambda t: t.transpose(1, 2).reshape(b, nc, G, hg, P, N)  # noqa: E731
    Z = (torch.exp(tot).float() * (h * dh).sum(-1).transpose(1, 2))[..., None]  # [b,nc,H,1]
    h, dh = back(h), back(dh)
    dh0 = torch.exp(tot[:, 0]).float()[..., None, None] * dh[:, 0].reshape(b, H, P, N) + g_loc[:, 0].reshape(b, H, P, N)
    # inside a chunk
    S = Cg @ Bg.transpose(-1, -2)  # [b,nc,G,1,Q,Q]
    Gm = dyh @ xh.transpose(-1, -2)  # [b,nc,G,hg,i,j]
    Lg = byg(L)
    M = S * Lg
    V = Bg @ dh.transpose(-1, -2)  # [b,nc,G,hg,Q,P]
    U = M.transpose(-1, -2) @ dyh + byg(w)[..., None] * V
    F = byg(w) * (xh * V).sum(-1)
    E = byg(e) * (dyh * (Cg @ h.transpose(-1, -2))).sum(-1)
    W = Gm * M
    direct = (W.sum(-2) + F).reshape(b, nc, H, Q)
    W = W * byg(dtc)[..., None, :] * (~torch.eye(Q, device=A.device, dtype=torch.bool))
    rows, cols = W.double().sum(-1).view(b, nc, H, Q), W.double().sum(-2).view(b, nc, H, Q)
    E, F = E.double().reshape(b, nc, H, Q), F.double().reshape(b, nc, H, Q) * dtc
    da = Z + (E + rows - cols).flip(-1).cumsum(-1).flip(-1) + F.cumsum(-1) - F
    ddt = (direct + A[:, None] * da).float()
    dA = (da * dtc).sum((0, 1, 3)).float()
    dS = (Gm * Lg * byg(dtc)[..., None, :]).sum(3)  # [b,nc,G,i,j]
    eh = (byg(e)[..., None] * dyh)
    dC = dS @ Bg[:, :, :, 0] + (eh @ h).sum(3)
    dB = dS.transpose(-1, -2) @ Cg[:, :, :, 0] + ((xh * wdt) @ dh).sum(3)
    dx = byg(dtc)[..., None] * U + s["D"].view(G, hg, 1, 1) * dyh
    dD = (s["dy"].float() * s["x"].float()).double().sum((0, 1, 3)).float()
    token = lambda t, *tail: t.reshape(b, nc * Q, *tail)[:, :T].contiguous()  # noqa: E731
    ddt = token(ddt.permute(0, 1, 3, 2), H)
    out = dict(dx=token(dx.permute(0, 1, 4, 2, 3, 5), H, P).to(io), dA=dA,
               dB=token(dB.permute(0, 1, 3, 2, 4), G, N).to(io), dC=token(dC.permute(0, 1, 3, 2, 4), G, N).to(io),
               dD=dD, dh0=dh0)
    if case["raw"]:
        ddt = ddt * (1.0 / (1.0 + torch.exp(-zr)))
        out["ddt_bias"] = ddt.double().sum((0, 1)).float()
    out["ddt"] = ddt
    return out


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    io = 2 if case["io"] == "bf16" else 4
    if case["op"] == "norm":
        n, res = case["rows"] * case["D"], 4 if case["res"] == "f32" else io
        if case["dir"] == "fwd":  # read x, residual; write out, r
            return {"bytes": n * (2 * io + 2 * res) + 4 * case["D"], "flops": 6 * n}
        return {"bytes": n * (2 * io + 3 * res) + 8 * case["D"], "flops": 14 * n}  # dout, r, dr_out; dx, dres
    if case["op"] == "gate":
        n = case["rows"] * case["D"]
        if case["dir"] == "fwd":  # read y, z; write out
            return {"bytes": 3 * n * io + 4 * case["D"], "flops": 12 * n}
        return {"bytes": 5 * n * io + 8 * case["D"], "flops": 30 * n}  # dout, y, z; dy, dz
    b, T, H, N, G, P = case["b"], case["T"], case["H"], case["N"], case["G"], 64
    tok, states = b * T, b * H * P * N * 4
    by = tok * H * P * io * 3 + tok * G * N * io * 4 + tok * H * 4 * 2 + 16 * H
    by += states * (1 + case["h0"] + case["dhf"])
    # the recurrence and its adjoint token by token: two state updates and four products with a state
    return {"bytes": by, "flops": 2 * tok * H * P * N * 6}


# ---------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    if case["op"] == "norm":
        return _exact_norm(case, d)
    if case["op"] == "gate":
        return _exact_gate(case, d)
    if case["b"] * case["H"] > 1024 or case["T"] > 8192:
        return None
    return _exact_ssd(case, d)


def _exact_norm(case, d):
    scale = case["scale"]
    if case["dir"] == "fwd":
        r = d["residual"] + scale * d["x"]
        return dict(out=r / torch.sqrt(r.pow(2).mean(1, keepdim=True) + 1e-5) * d["weight"], r=r)
    r, go = d["r"], d["dout"]
    m = r.pow(2).mean(1, keepdim=True) + 1e-5
    # out_c = w_c r_c m^-1/2, dm/dr_k = 2 r_k / D
    dm = (go * d["weight"] * r).sum(1, keepdim=True) * -0.5 * m.pow(-1.5)
    dr = go * d["weight"] * m.pow(-0.5) + dm * 2.0 * r / case["D"] + d["dr_out"]
    return dict(dx=dr * scale, dres=dr, dw=(go * r * m.pow(-0.5)).sum(0))


def _exact_gate(case, d):
    D, n = case["D"], case["groups"]
    y, z = d["y"], d["z"]
    sg = torch.sigmoid(z)
    silu = z * sg
    dsilu = sg + silu * (1 - sg)
    first = case["order"] == "norm_first"
    q = (y if first else y * silu).reshape(-1, D // n)
    m = q.pow(2).mean(1, keepdim=True) + 1e-5
    w = d["weight"].view(1, n, D // n).expand(case["rows"], -1, -1).reshape(-1, D // n)
    if case["dir"] == "fwd":
        o = (q / torch.sqrt(m) * w).view(-1, D)
        return dict(out=o * silu if first else o)
    go = d["dout"]
    t = (go * silu if first else go).reshape(-1, D // n)
    dm = (t * w * q).sum(1, keepdim=True) * -0.5 * m.pow(-1.5)
    dq = (t * w / torch.sqrt(m) + dm * 2.0 * q / (D // n)).view(-1, D)
    dw = (t * q / torch.sqrt(m)).view(-1, D).sum(0)
    if first:
        return dict(dy=dq, dz=go * (q / torch.sqrt(m) * w).view(-1, D) * dsilu, dw=dw)
    return dict(dy=dq * silu, dz=dq * y * dsilu, dw=dw)


def _exact_ssd(case, d, block=64):
    """Token by token: h_t = e_t h_{t-1} + dt_t x_t B_t^T, y_t = h_t C_t + D x_t, and the adjoint
    lam_t = dy_t C_t^T + e_{t+1} lam_{t+1}; the states of `block` tokens are kept at a time."""
    b, T, H, N, G, P = case["b"], case["T"], case["H"], case["N"], case["G"], 64
    hg = H // G
    x, dy, A = d["x"], d["dy"], d["A"]
    dt = d["dt"]
    if case["raw"]:
        dt = torch.nn.functional.softplus(dt + d["dt_bias"], threshold=200.0)
    ex = torch.exp(dt * A)
    head = lambda t: t.repeat_interleave(hg, 1)  # [b,G,N] -> [b,H,N]  # noqa: E731
    h = d["h0"].clone() if d["h0"] is not None else torch.zeros(b, H, P, N, dtype=torch.float64, device=x.device)

    def step(h, t):
        u = (dt[:, t, :, None] * x[:, t])[..., None]
        return torch.addcmul(h * ex[:, t, :, None, None], u, head(d["B"][:, t])[:, :, None, :])

    marks = []
    for t in range(T):
        if t % block == 0:
            marks.append(h)
        h = step(h, t)
    dx, ddt = torch.empty_like(x), torch.empty_like(dt)
    dB, dC = torch.empty_like(d["B"]), torch.empty_like(d["C"])
    dA = torch.zeros(H, dtype=torch.float64, device=x.device)
    lam = d["dh_final"].clone() if d["dh_final"] is not None else torch.zeros_like(h)
    for k in range(len(marks) - 1, -1, -1):
        hs = [marks[k]]
        for t in range(k * block, min(T, (k + 1) * block)):
            hs.append(step(hs[-1], t))
        for t in range(min(T, (k + 1) * block) - 1, k * block - 1, -1):
            ht, hp = hs[t - k * block + 1], hs[t - k * block]
            Bt, Ct, xt, gy = head(d["B"][:, t]), head(d["C"][:, t]), x[:, t], dy[:, t]
            dC[:, t] = (gy[:, :, None, :] @ ht)[:, :, 0].view(b, G, hg, N).sum(2)
            lam = torch.addcmul(lam, gy[..., None], Ct[:, :, None, :])
            lB = (lam @ Bt[..., None])[..., 0]  # [b,H,P]
            dx[:, t] = dt[:, t, :, None] * lB + d["D"][:, None] * gy
            dB[:, t] = (dt[:, t, :, None] * (xt[:, :, None, :] @ lam)[:, :, 0]).view(b, G, hg, N).sum(2)
            lam_in = lam * ex[:, t, :, None, None]
            da = (lam_in * hp).sum((2, 3))
            ddt[:, t] = (xt * lB).sum(2) + A * da
            dA += (dt[:, t] * da).sum(0)
            lam = lam_in
    out = dict(dx=dx, dA=dA, dB=dB, dC=dC, dD=(x * dy).sum((0, 1, 3)), dh0=lam)
    if case["raw"]:
        ddt = ddt * torch.sigmoid(d["dt"] + d["dt_bias"])
        out["ddt_bias"] = ddt.sum((0, 1))
    out["ddt"] = ddt
    return out
