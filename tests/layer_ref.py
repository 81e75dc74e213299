"""Definitions in 64 bits of the operators of include/forge_layer.h, on CPU tensors."""
import torch

F64 = torch.float64
U = 2.0 ** -24  # half a step of fp32, relative


def norm_h(x, residual):
    """The stored stream: the fp32 sum rounded to the dtype of x."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def norm(h, gain, eps):
    h, gain = h.to(F64), gain.to(F64)
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * gain, rstd


def norm_grads(dy, h, gain, rstd, dh=None):
    dy, h, gain, rstd = (t.to(F64) for t in (dy, h, gain, rstd))
    a, s = dy * gain, rstd[:, None]
    dx = s * a - h * s ** 3 * (a * h).mean(1, keepdim=True)
    if dh is not None:
        dx = dx + dh.to(F64)
    return dx, (dy * h * s).sum(0)


def spans(ends, T):
    """Row ranges of the groups, and of the rows after them."""
    out, at = [], 0
    for e in ends:
        e = min(max(int(e), at), T)
        out.append((at, e))
        at = e
    return out, (at, T)


def grouped(A, W, ends, transposed):
    """A_e W_e^T (transposed) or A_e W_e by group in 64 bits, and the sums of magnitudes."""
    groups, rest = spans(ends, A.shape[0])
    A, W = A.to(F64), W.to(F64)
    out = torch.zeros(A.shape[0], W.shape[1] if transposed else W.shape[2], dtype=F64)
    mag = torch.zeros_like(out)
    for e, (a, b) in enumerate(groups):
        w = W[e].t() if transposed else W[e]
        out[a:b], mag[a:b] = A[a:b] @ w, A[a:b].abs() @ w.abs()
    return out, mag


def grouped_wgrad(X, dY, ends):
    groups, _ = spans(ends, X.shape[0])
    X, dY = X.to(F64), dY.to(F64)
    return torch.stack([dY[a:b].t() @ X[a:b] for a, b in groups])


def adamw(w, g, m, v, hyper, step):
    """One step in 64 bits from the 32-bit hyper-parameters."""
    f = lambda k: float(torch.tensor(hyper[k], dtype=torch.float32))  # noqa: E731
    w, g, m, v = (t.to(F64) for t in (w, g, m, v))
    m = f("beta1") * m + (1 - f("beta1")) * g
    v = f("beta2") * v + (1 - f("beta2")) * g * g
    mh, vh = m / (1 - f("beta1") ** step), v / (1 - f("beta2") ** step)
    return w - f("lr") * (f("weight_decay") * w + mh / (vh.sqrt() + f("eps"))), m, v
