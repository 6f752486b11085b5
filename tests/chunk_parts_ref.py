"""The chunked delta rule of one sequence and head as the tensor-core path computes it, in fp32 on the CPU, with a chosen number of bf16
parts of what is fp32: a model of that path's precision, apart from its kernels.
"""
import torch

CHUNK = 64


def parts(x, n):
    out = []
    for _ in range(n):
        out.append(x.bfloat16().float())
        x = x - out[-1]
    return out


def product(a, b, na, nb):
    """a @ b by parts, the small products first; 1 part where a factor is exact in bf16."""
    a, b = parts(a.float(), na), parts(b.float(), nb)
    n = max(na, nb)
    terms = [a[o - q] @ b[q] for o in range(n - 1, -1, -1) for q in range(o + 1) if o - q < na and q < nb]
    acc = terms[0]
    for t in terms[1:]:
        acc = acc + t
    return acc


def delta(q, k, v, g, beta, h0, scale, dy, dh, n):
    """h_final, dh0, dg, dbeta with `n` parts; q, k [L, N], v, dy [L, P] bf16, the others fp32."""
    L = q.shape[0]
    chunks, states, X, out = [], [h0], dh, {"dg": torch.zeros(L), "dbeta": torch.zeros(L)}
    for t0 in range(0, L, CHUNK):
        s = slice(t0, min(L, t0 + CHUNK))
        qc, kc, b = q[s].float(), k[s].float(), beta[s]
        m = len(b)
        G = g[s].double().cumsum(0)
        D = torch.exp((G[:, None] - G).masked_fill(~torch.ones(m, m).tril().bool(), -torch.inf)).float()
        low = (kc @ kc.T) * D * torch.ones(m, m).tril(-1)
        x = torch.linalg.solve_triangular(torch.eye(m) + low * b, low, upper=False)
        A = scale * D * (qc @ kc.T)
        grow, fade, last = torch.exp(G).float(), torch.exp(G[-1] - G).float(), torch.exp(G[-1]).float()
        H = states[-1]
        R = v[s].float().T - product(H.T, kc.T, n, 1) * grow
        e = product(R, (torch.eye(m) - x * b).T, n, n)
        u = b * e
        y = scale * product(H.T, qc.T, n, 1) * grow + product(u, A.T, n, n)
        states.append((last * H.T + product(u * fade, kc, n, 1)).T)
        chunks.append((s, torch.eye(m) - b[:, None] * x, A, grow, fade, last, e, y))
    for i in range(len(chunks) - 1, -1, -1):
        s, Tb, A, grow, fade, last, e, y = chunks[i]
        b, dyc = beta[s], dy[s].float().T
        end = (X * states[i + 1]).sum()
        dU = product(X.T, k[s].float().T, n, 1) * fade + product(dyc, A, 1, n)
        du = product(dU, Tb, n, n)
        local = (dyc * y).sum(0) - b * (du * v[s].float().T).sum(0)
        out["dg"][s] = (end.double() + local.double().flip(0).cumsum(0).flip(0)).float()
        out["dbeta"][s] = (du * e).sum(0)
        X = (last * X.T + product(scale * dyc * grow, q[s].float(), n, 1) - product(b * du * grow, k[s].float(), n, 1)).T
    return {"h_final": states[-1], "dh0": X, **out}
