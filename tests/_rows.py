"""What the tests of the row operators share: definitions in 64 bits and the
rounding errors that the formulas allow (U is half a step of fp32)."""
import torch

U = 2.0**-24
FLOATS = (torch.float32, torch.bfloat16, torch.float16)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def rounded(value, dtype):
    """The error of one rounding of ``value`` to the type."""
    return value.abs() * half_step(dtype) * 1.001 + tiny(dtype)


def assert_close(got, want, tol, what=""):
    got, want = got.detach().double().cpu(), want.detach().double().cpu()
    assert got.shape == want.shape, "%s: %s, not %s" % (what, tuple(got.shape), tuple(want.shape))
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    bad = ~(same | ((got - want).abs() <= tol.cpu()))
    assert not bad.any(), "%s: %d of %d values off, first at %s: %r, not %r within %r" % (
        what, int(bad.sum()), bad.numel(), torch.nonzero(bad)[0].tolist(), got[bad][0].item(), want[bad][0].item(),
        torch.broadcast_to(tol.cpu(), bad.shape)[bad][0].item())


def scores(T, V, dtype, seed, spread=2.0, pad=0, device="cuda"):
    """Rows of logits, a few well above the others, in rows ``pad`` longer than they are used."""
    gen = torch.Generator().manual_seed(seed)
    z = spread * torch.randn(T, V, generator=gen)
    at = torch.randint(V, (T, min(V, 4)), generator=gen)
    z.scatter_(1, at, 6 + 3 * torch.randn(at.shape, generator=gen))
    rows = torch.full((T, V + pad), float("nan"))
    rows[:, :V] = z
    return rows.to(dtype).to(device)[:, :V]


class Softmax:
    """A row's distribution in 64 bits, and how far sums in fp32 may be from it."""

    def __init__(self, logits, temperature):
        z = logits.detach().double().cpu()
        V = z.shape[-1]
        self.temperature = temperature
        self.m = z.max(-1, keepdim=True).values
        self.empty = self.m == -torch.inf
        self.d = torch.where(self.empty, -torch.inf, (z - self.m) / temperature)
        e = self.d.exp()
        self.log_s = e.sum(-1, keepdim=True).log()
        self.lp = self.d - self.log_s
        # an fp32 result past the type's largest value is an infinity by rounding to nearest: (lowest - m) / 0.5 is
        self.lp = torch.where(self.empty | (self.lp < -torch.finfo(torch.float32).max), -torch.inf, self.lp)
        self.p = torch.where(self.empty, 0.0, self.lp.exp())
        self.size = torch.where(self.p > 0, -self.d, 0.0)  # |d| of what counts
        self.entropy = -torch.where(self.p > 0, self.p * torch.where(self.p > 0, self.lp, 0.0), 0.0).sum(-1)
        # log s: each term's exponent is off by 3 U |d| (the difference, its factor, the factor's own rounding) and
        # 4 U of the exponential and its sum of a vector; a thread's sums take V / (64 * 4) additions at most, their
        # join 12, and the change to the row's reference, up to 24 powers of two and 17 in natural units, 3 U of it
        self.depth = V / 256 + 12 + 4 + 3 * 17
        mean = (self.p * self.size).sum(-1, keepdim=True)
        square = (self.p * self.size**2).sum(-1, keepdim=True)
        self.tol_log_s = U * (3 * mean + self.depth + 3 * torch.where(self.empty, 0.0, self.log_s.abs()))
        # entropy: log s, and sum of p d whose terms are off by their exponent's error, two more roundings and the
        # sums' depth; the change of reference adds s times the step, twice, which cancels
        self.tol_entropy = (self.tol_log_s + U * (3 * square + (self.depth + 6) * mean + 4 * 17 + self.entropy[..., None]))[..., 0]

    def tol_lp(self, d, lp):
        """Of (x - m) / temperature - log s."""
        fin = torch.isfinite(d) & torch.isfinite(lp)
        return self.tol_log_s + U * torch.where(fin, 3 * d.abs() + lp.abs(), 0.0)

    def relative(self):
        """Relative error of every p from fp32 sums: its exponent's, and two roundings of the exponential."""
        log_s = torch.where(self.empty, 0.0, self.log_s.abs())
        return self.tol_log_s + U * (4 * self.size + 3 * log_s + 4)
