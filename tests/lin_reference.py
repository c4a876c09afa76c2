"""Decayed linear attention in 64 bits, token by token, with the absolute sums that bound its rounding errors.

For S_t = a_t S_{t-1} + k_t v_t^T and o_t = S_t^T q_t the companions |S|_t = a_t |S|_{t-1} + |k_t| |v_t|^T and
B_t = |S|_t^T |q_t| bound every partial sum, whatever its order: a result whose terms each carry a relative
error of at most e is off by at most e B_t (e |S|_t for the state).
"""
import torch

LOG_MIN = -120.0


def run(q, k, v, la, cu, init, ckpt_stride=0):
    """(o, B, final, |final|, checkpoints, |checkpoints|) in 64 bits on the inputs' device; la [T, H] or [H]."""
    T, H = v.shape[0], v.shape[1]
    per = H // q.shape[1]
    q, k, v = (x.double() for x in (q, k, v))
    q, k = q.repeat_interleave(per, 1), k.repeat_interleave(per, 1)
    la = (la if la.dim() == 2 else la.expand(T, H)).double()
    a = torch.where(la >= LOG_MIN, la, torch.full_like(la, float("-inf"))).exp()   # NaN too
    o, b = torch.zeros_like(v), torch.zeros_like(v)
    fin, afin, ck, ack = [], [], [], []
    cu = cu.tolist()
    for i in range(len(cu) - 1):
        S = torch.zeros(H, q.shape[2], v.shape[2], dtype=torch.float64, device=q.device) if init is None else init[i].double()
        A = S.abs()
        for t in range(cu[i], cu[i + 1]):
            S = a[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            A = a[t][:, None, None] * A + k[t].abs()[:, :, None] * v[t].abs()[:, None, :]
            o[t] = torch.einsum("hd,hde->he", q[t], S)
            b[t] = torch.einsum("hd,hde->he", q[t].abs(), A)
            if ckpt_stride and (t + 1 - cu[i]) % ckpt_stride == 0:
                ck.append(S)
                ack.append(A)
        fin.append(S)
        afin.append(A)
    st = lambda x: torch.stack(x) if x else torch.zeros(0, H, q.shape[2], v.shape[2], dtype=torch.float64, device=q.device)  # noqa: E731
    return o, b, st(fin), st(afin), st(ck), st(ack)


def f32_factor(tokens, dk):
    """Relative error of an fp32 sum formed over `tokens` tokens and dk channels, as a factor of B or |S|: at most
    one rounding a token and channel and a few for each weight (an exponential of an argument of at most 120 in
    magnitude that was rounded once is off by 120 half steps, its own error by two), each of half a step, twice
    that where an accumulator truncates."""
    return 2 * (tokens + dk + 130) * 2.0 ** -24


def o_tolerance(o, b, dtype, tokens, dk):
    """Element-wise bound for o: bf16 rounds each score or state element once and the result once (half a step is
    2^-8 of the value), on top of the fp32 sums; fp32 has those alone."""
    f = f32_factor(tokens, dk)
    if dtype == torch.bfloat16:
        return (2.0 ** -8 + 2.0 ** -16 + f) * b * (1 + 2.0 ** -8) + 2.0 ** -8 * o.abs() + 1e-30
    return f * b + 1e-30


def check(name, got, want, tol):
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), f"{name}: non-finite values"
    over = err > tol
    assert not over.any(), f"{name}: {int(over.sum())} of {over.numel()} values off, worst {float((err / tol).max()):.3g} of the bound"
