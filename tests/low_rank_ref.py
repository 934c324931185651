"""Newton-Schulz steps on matrices of low rank: the 64-bit result and how far a
kernel's may be from it, both from the singular values (CPU tensors).

The steps act on the squares l of the singular values, O = Q X with Q a
polynomial of G = X X^T: q(l) is formed value by value, with l >= 0 throughout,
so that nothing here grows that the steps in exact arithmetic would not."""
import torch

U = 2.0 ** -24
QUINTIC = (3.4445, -4.7750, 2.0315)
COEFFICIENTS = (QUINTIC, (2.0, -1.5, 0.5), (1.5, -0.5, 0.0))


def low_rank(seed, rows, cols, rank, dt, whole=True):
    """A product of two factors: of small whole numbers, which makes every element exact in bf16
    (the rank is what it says in either type), or of normal values, then rounded."""
    g = torch.Generator().manual_seed(seed)
    if whole:
        top = 4 if rank <= 32 else 2 if rank <= 128 else 1
        left = torch.randint(-1, 2, (rows, rank), generator=g).double()
        right = torch.randint(-top, top + 1, (rank, cols), generator=g).double()
        M = left @ right
        assert float(M.abs().max()) <= 256 and torch.equal(M.to(dt).double(), M)
        return M.to(dt)
    return (torch.randn(rows, rank, generator=g) @ torch.randn(rank, cols, generator=g)).to(dt)


class Steps:
    """The singular values and vectors of one matrix, for any number of steps on it."""

    def __init__(self, M, eps=1e-7):
        X = M.double()
        self.tall = X.shape[0] > X.shape[1]
        self.X = X.T if self.tall else X
        norm = float(torch.linalg.vector_norm(self.X))
        self.size = norm + float(torch.tensor(eps, dtype=torch.float32))
        self.share = norm / self.size
        self.W, self.s, self.V = torch.linalg.svd(self.X / self.size, full_matrices=False)

    def run(self, steps, coefficients, least=1e-12):
        """(O, bound of |O' - O|_F in fp32 outputs, without what U itself is off by)."""
        a, b, c = (float(torch.tensor(v, dtype=torch.float32)) for v in coefficients)
        first = self.s ** 2
        q, dq, l, dl = (torch.ones_like(first), torch.zeros_like(first), first.clone(),
                        torch.ones_like(first))
        for _ in range(steps):
            p, dp = a + b * l + c * l * l, (b + 2 * c * l) * dl
            q, dq = q * p, dq * p + q * dp
            l, dl = l * p * p, dl * p * p + 2 * l * p * dp
        O = self.W @ torch.diag(self.s * q) @ self.V
        n, length = self.X.shape
        # The product at the end, of three bf16 numbers an operand: 24 bits of Q and X, what the
        # planes left out make, 4 u together; and six products of n values in fp32 sums, at least
        # eight at a time: 6 n / 8 roundings of at most u (|Q| |X|), of either sign, so that over a
        # matrix they add up to the root of their number.
        Q = (self.W * q) @ self.W.T / self.size
        end = (4 + (6 * n / 8) ** 0.5) * U * float(torch.linalg.vector_norm(Q.abs() @ self.X.abs()))
        # The n x n part in 64 bits: a change D of G moves O by q[l_i, l_j] D_ij s_j (divided
        # differences, in G's own basis).  The roundings of G, P and Q of a step, and what keeps
        # G positive, are (16 + 4 n) 2^-53 |G| at most, and more by the root of a long side's sums.
        away = (first[:, None] - first[None, :]).abs() > 1e-7 * (first[:, None] + first[None, :])
        gap = torch.where(away, first[:, None] - first[None, :], torch.ones(1, dtype=torch.float64))
        divided = torch.where(away, (q[:, None] - q[None, :]) / gap, (dq[:, None] + dq[None, :]) / 2)
        D = (16 + 4 * n) * 2.0 ** -53 * max(1.0, length ** 0.5 / 64) * float((first ** 2).sum().sqrt())
        inner = steps * D * float((divided.abs() * self.s[None, :]).max())
        return O.T if self.tall else O, end + inner + least

    def steepest(self, steps, coefficients):
        """The largest |f'| on [0, 1] of what the steps make of a singular value."""
        a, b, c = coefficients
        s = torch.linspace(0, 1, 20001, dtype=torch.float64)
        d = torch.ones_like(s)
        for _ in range(steps):
            d, s = d * (a + 3 * b * s ** 2 + 5 * c * s ** 4), a * s + b * s ** 3 + c * s ** 5
        return float(d.abs().max())
