"""How large the rounding errors of the prefill's gradients are in the 2-norm: every gradient is a sum of
products over token pairs and state entries whose roundings are independent of one another, so its error
is a small multiple of a step times the root of the sum of the terms' squares.

`spread` evaluates those roots, the recurrence and its adjoint (tests/backward_ref.py) on squares:
h2_t = e_t^2 h2_{t-1} + (dt_t x_t B_t^T)^2, and so on.  da's terms reach dA through many tokens at
once, so dA takes the sum of dt_t times da_t's root instead of the root of a sum.
`limits` turns them into bounds on ||got - ref||, with u = 2^-24, v = 2^-8:
  tensor cores, fp32 results   a term has at most four factors carried in 16 bits (2^-16 each, two bf16
                               halves): 4 * 2^-16
  bf16 results                 besides, roundings to bf16 of at most half a step v each, v / sqrt(3) in the mean
                               square, independent: the result's own, and on the tensor cores one factor in
                               dx (the pair terms), two in dB and dC (weighted row and state); 1.25 times that,
                               as the smallest gradients have 64 elements
  fp32 path                    three products in a row of at most 128 terms each, whose running sums take
                               a rounding a term: 3 sqrt(128) u < 34 u; decays 2 ulp and |c| u in the exponent
                               c, where e^c leaves |c| <= 16 to count: 18 u a factor, two of them; a scan
                               step of 2 u a chunk of 64: (70 + 2 chunks) u
  all                          a decay below 2^-126 (1.2e-38) may come out as zero: 1e-30 an element, which is that
                               times operands of up to 1e7
"""
import torch

U, V = 2.0 ** -24, 2.0 ** -8


def spread(dy, x, dt, A, B, C, D, h0=None, dhf=None):
    v = [None if t is None else t.double() for t in (dy, x, dt, A, B, C, D, h0, dhf)]
    ex2 = torch.exp(2 * v[2] * v[3])
    dta = v[2].abs()
    dy, x, dt, A, B, C, D, h0, dhf = [None if t is None else t.square() for t in v]
    b, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    hg = H // G
    Bh, Ch = B.repeat_interleave(hg, 2), C.repeat_interleave(hg, 2)
    zero = torch.zeros(b, H, P, N, dtype=torch.float64, device=x.device)
    hs = [zero if h0 is None else h0]
    for t in range(T):
        hs.append(ex2[:, t, :, None, None] * hs[-1] + (dt[:, t, :, None] * x[:, t])[..., None] * Bh[:, t, :, None, :])
    lam = zero if dhf is None else dhf
    out = dict(dx=torch.zeros_like(x), ddt=torch.zeros_like(dt), dB=torch.zeros_like(B), dC=torch.zeros_like(C),
               da=torch.zeros_like(dt))
    for t in range(T - 1, -1, -1):
        lam = lam + dy[:, t, :, :, None] * Ch[:, t, :, None, :]
        lB = (lam * Bh[:, t, :, None, :]).sum(-1)
        out["dx"][:, t] = dt[:, t, :, None] * lB + D[:, None] * dy[:, t]
        out["dB"][:, t] = (dt[:, t, :, None] * (lam * x[:, t, :, :, None]).sum(2)).view(b, G, hg, N).sum(2)
        out["dC"][:, t] = (hs[t + 1] * dy[:, t, :, :, None]).sum(2).view(b, G, hg, N).sum(2)
        lam = ex2[:, t, :, None, None] * lam
        out["da"][:, t] = (lam * hs[t]).sum((2, 3))
        out["ddt"][:, t] = (x[:, t] * lB).sum(-1) + A * out["da"][:, t]
        hs.pop()
    out = {k: t.sqrt() for k, t in out.items()}
    out["dA"] = (dta * out["da"]).sum((0, 1))
    out["dD"] = (x * dy).sum((0, 1, 3)).sqrt()
    out["dh0"] = lam.sqrt()
    return out


def limits(sp, ref, T, io, tc):
    """Bounds on the 2-norm of each gradient's error.  io: the type of x; tc: on the tensor cores."""
    f = 4 * 2.0 ** -16 if tc else (70 + 2 * -(-T // 64)) * U
    out = {k: f * sp[k].norm().item() + 1e-30 * sp[k].numel() ** 0.5 for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dh0")}
    if io == torch.bfloat16:
        for k, n in (("dx", 1), ("dB", 2), ("dC", 2)):
            out[k] += 1.25 * V * ((n * tc * sp[k].square().sum() + ref[k].square().sum()) / 3).sqrt().item()
    return out
