"""The SSD recurrence and its adjoint token by token in 64 bits (torch, any device), and the
magnitudes of the sums behind every gradient.

h_t = e_t h_{t-1} + dt_t x_t B_t^T, y_t = h_t C_t + D x_t with e_t = exp(dt_t A); with lam_t the
adjoint of h_t, lam_t = dy_t C_t^T + e_{t+1} lam_{t+1}:
  dx_t = dt_t lam_t B_t + D dy_t, dB_t = dt_t lam_t^T x_t, dC_t = h_t^T dy_t (summed over a group's heads),
  da_t = <e_t lam_t, h_{t-1}>, ddt_t = x_t . lam_t B_t + A da_t, dA = sum dt_t da_t, dh0 = e_0 lam_0.
"""
import torch


def step_gradients(dy, x, dt, A, B, C, D, h0=None, dhf=None, absolute=False):
    """Gradients by name, as float64; also "da" [b,T,H] and "y".  With absolute=True every factor
    but the decays is taken by its absolute value: the magnitudes."""
    v = [None if t is None else t.double() for t in (dy, x, dt, A, B, C, D, h0, dhf)]
    if absolute:
        ex = torch.exp(v[2] * v[3])
        v = [None if t is None else t.abs() for t in v]
    dy, x, dt, A, B, C, D, h0, dhf = v
    if not absolute:
        ex = torch.exp(dt * A)
    b, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    hg = H // G
    Bh, Ch = B.repeat_interleave(hg, 2), C.repeat_interleave(hg, 2)
    zero = torch.zeros(b, H, P, N, dtype=torch.float64, device=x.device)
    hs = [zero if h0 is None else h0]
    for t in range(T):
        hs.append(ex[:, t, :, None, None] * hs[-1] + (dt[:, t, :, None] * x[:, t])[..., None] * Bh[:, t, :, None, :])
    lam = zero if dhf is None else dhf
    out = dict(dx=torch.zeros_like(x), ddt=torch.zeros_like(dt), dB=torch.zeros_like(B), dC=torch.zeros_like(C),
               da=torch.zeros_like(dt), y=torch.zeros_like(x))
    for t in range(T - 1, -1, -1):
        out["y"][:, t] = (hs[t + 1] * Ch[:, t, :, None, :]).sum(-1) + D[:, None] * x[:, t]
        lam = lam + dy[:, t, :, :, None] * Ch[:, t, :, None, :]
        lB = (lam * Bh[:, t, :, None, :]).sum(-1)
        out["dx"][:, t] = dt[:, t, :, None] * lB + D[:, None] * dy[:, t]
        out["dB"][:, t] = (dt[:, t, :, None] * (lam * x[:, t, :, :, None]).sum(2)).view(b, G, hg, N).sum(2)
        out["dC"][:, t] = (hs[t + 1] * dy[:, t, :, :, None]).sum(2).view(b, G, hg, N).sum(2)
        lam = ex[:, t, :, None, None] * lam
        da = (lam * hs[t]).sum((2, 3))
        out["da"][:, t] = da
        out["ddt"][:, t] = (x[:, t] * lB).sum(-1) + A * da
    out["dA"] = (dt * out["da"]).sum((0, 1))
    out["dD"] = (x * dy).sum((0, 1, 3))
    out["dh0"] = lam
    return out
