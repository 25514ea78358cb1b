"""The chunk form of the gated delta rule in fp32 numpy, as the bf16 kernels run it: what was computed enters
a product as the sum of `planes[name]` bf16 numbers, by the name of the operand.  For the test suite only: it
shows what the checks of the kernels' precision can tell apart."""
import numpy as np
import torch

from tests.delta_helpers import delta_case

F = np.float32
C = 64
# operands that were computed: forwards the inverse, X, the state met by the keys, leave beta E (fp32 results);
# backwards the inverse, P, beta dU, the state's gradient, -enter dX and scale enter dO; for the gradient of
# the gates the states and their gradients at the chunks, dX and E
FORWARD = ("inverse", "x", "state", "w")
BACKWARD = ("inverse_t", "p_t", "u_t", "dstate", "w_t", "q_t")
GATES = ("before", "after", "dx", "err")


def rounded(x, planes):
    """x as the sum of `planes` bf16 numbers, largest first."""
    left, out = torch.from_numpy(np.ascontiguousarray(x, F)), torch.zeros(x.shape)
    for _ in range(planes):
        p = left.bfloat16().float()
        out, left = out + p, left - p
    return out.numpy()


def head(q, k, v, g, beta, S, scale, do, dS, planes=None):
    """One head's sequence (L, K), (L, V), (L,): the final state, and the gradients of the first one and of g
    (with the size that its error goes by: the root of the sum of the squares of what is added up in it)."""
    at = lambda name, x: rounded(x, (planes or {}).get(name, 3))  # noqa: E731
    L, kept = len(g), []
    dg, size = np.empty(L), np.empty(L)
    for c in range(0, L, C):
        kc, qc, vc, b = k[c:c + C], q[c:c + C], v[c:c + C], beta[c:c + C, None]
        G = np.cumsum(g[c:c + C].astype(np.float64))
        D = np.tril(np.exp((G[:, None] - G[None]).astype(F)))
        enter, leave, through = np.exp(G.astype(F))[:, None], np.exp((G[-1] - G).astype(F))[:, None], F(np.exp(G[-1]))
        B = np.tril(D * (kc @ kc.T), -1)
        A = B * b.T
        inv = np.eye(len(kc), dtype=F)
        for t in range(1, len(kc)):
            inv[t, :t] = -(A[t, :t] @ inv[:t, :t])
        x = vc - enter * (kc @ at("state", S))
        e = at("inverse", inv) @ at("x", x)
        kept.append((kc, qc, b, enter, leave, through, inv, F(scale) * D * (qc @ kc.T), B, e, S))
        S = through * S + kc.T @ at("w", leave * b * e)
    for c, (kc, qc, b, enter, leave, through, inv, P, B, e, before) in zip(reversed(range(0, L, C)), reversed(kept)):
        d, after = do[c:c + C], dS
        du = at("p_t", P.T) @ d + leave * (kc @ at("dstate", dS))
        dx = at("inverse_t", inv.T) @ at("u_t", b * du)
        dS = through * dS + qc.T @ at("q_t", F(scale) * enter * d) - kc.T @ at("w_t", enter * dx)
        bf, ef = at("before", before), at("err", e)
        Z = np.tril(d @ ef.T) * b.T * P - np.tril(at("dx", dx) @ ef.T, -1) * b.T * B
        parts = [qc * (F(scale) * enter * (d @ bf.T)), -kc * (enter * (at("dx", dx) @ bf.T)),
                 -kc * (leave * b * (ef @ at("after", after).T))]
        met = through * (before * after)
        dG = sum((Z.sum(1), -Z.sum(0), *(x.sum(1) for x in parts))).astype(np.float64)
        dG[-1] += met.sum() - parts[2].sum()
        squares = sum(((Z ** 2).sum(1), (Z ** 2).sum(0), *((x ** 2).sum(1) for x in parts))).astype(np.float64)
        squares[-1] += (met ** 2).sum() + (parts[2] ** 2).sum()
        dg[c:c + C], size[c:c + C] = np.cumsum(dG[::-1])[::-1], np.cumsum(squares[::-1])[::-1] ** 0.5
    return dict(h_final=S, dh0=dS, dg=dg), size


def off(got, want, L, size, units=16):
    """A head's error in the 2-norm as a share of what it may be.  A result is a sum that goes through at most
    four products a chunk; an fp32 product of 24-bit operands is off, in the 2-norm, by the operands' roundings
    and those of its sums, which have either sign and add up as their squares: 2 u for each of the two operands
    and 4 u for up to 16 partial sums of half a unit each, so sqrt(4 (2^2 + 2^2 + 4^2)) < 10 u a chunk, and the
    chunks' errors as their squares too.  16 u, as a state is one summand beside the chunk's.  For dg, whose
    size counts every term of its sums in full where their errors partly cancel, 5 u."""
    error = np.linalg.norm(np.asarray(got, np.float64) - want)
    return error / (units * 2.0 ** -24 * np.sqrt(-(-L // C)) * np.linalg.norm(size))


DG_UNITS = 5


# B, L, Hk, H, K, V: long memories and keys that meet again, so that every product's part is a large one
SHAPES = [(2, 128, 1, 2, 16, 32), (1, 192, 2, 2, 64, 64), (2, 130, 2, 4, 72, 40)]


def case(B, L, Hk, H, K, V):
    """Inputs of a call on the CPU, and the gradients that enter its backward."""
    k = delta_case(B, L, Hk, H, K, V, torch.bfloat16, seed=K, l2norm=True, device="cpu", beta=2.0)
    k["g"] = 0.02 * k["g"]
    n = torch.Generator().manual_seed(K + 1)
    return k, torch.randn(B, L, H, V, generator=n).bfloat16(), 0.3 * torch.randn(B, H, K, V, generator=n)
