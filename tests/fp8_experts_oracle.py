"""The FP8 experts in fp64 from their definition, how near a forward pass has to come in the 2-norm, and
passes with a mistake in them, which have to be told from the right one (test infrastructure; nothing here is
shared with the library).

The bound. A forward pass is off by
  - the rounding of out to bf16: at most 2^-8 / sqrt(3) = 0.00226 in the 2-norm (evenly spread errors of values
    just above a power of two);
  - codes of h that come out as their neighbour, because h itself is off. With d_i the error of h_i and s_i the
    step between the codes around it, a border lies in between with probability d_i / s_i and costs s_i, so
    that the squares add to sum d_i s_i on average. s_i is |h_i| / 8 at most, so that is at most |d| |h| / 8. g
    and u are off by 2.6e-5 at most in the 2-norm (the cut of the FP8 matrix units, include/moe_fp8.h), h by up
    to twice that: sqrt(2 * 2.6e-5 / 8) = 0.00255 of h, and of out, as W2 spreads h's errors as it does h;
  - the cut in the second product, 2.6e-5.
Together 0.0034 on average. Over some 30000 values of h about 30 codes move, so that their squares' sum stays well
within 3 times its average, and the whole within sqrt(0.00226^2 + 3 * 0.00255^2) = 0.00496: BOUND is 0.005.
Kernels that sum in fp32 are off by 1e-6 in g and u and move next to no codes, at any size:
sqrt(2 * 1e-6 / 8) = 0.0005 of h, and sqrt(0.00226^2 + 3 * 0.0005^2) = 0.00242 the whole; FP32_SUMS is 0.00245.
A single token may have two of its largest steps more."""
import torch

from tests import fp8_oracle as o

F64 = torch.float64
BOUND = 0.005
FP32_SUMS = 0.00245


def inputs(T, H, I, E, total, k, base, seed, device="cpu"):
    """x, ids, weights, (codes, scales) of w13 and of w2. Ids lie in [0, total)."""
    g = torch.Generator(device).manual_seed(seed)
    like = dict(generator=g, device=device)
    x = torch.randn((T, H), **like).bfloat16()
    ids = torch.rand((T, total), **like).argsort(dim=1)[:, :k].int().contiguous()
    weights = torch.rand((T, k), **like) + 0.1

    def matrices(rows, width):
        codes = (torch.randn((E, rows, width), **like) * 90).clamp(-448, 448).to(torch.float8_e4m3fn)
        return codes, (torch.rand((E, rows // 128, width // 128), **like) + 0.5) * (width ** -0.5 / 90)
    return x, ids, weights, matrices(2 * I, H), matrices(H, I)


def forward(x, ids, weights, w13, w2, base, mistake=None):
    """(out fp64 [T, H], the largest cost of a moved code for each token). mistake: a name of MISTAKES."""
    (T, H), E, I = x.shape, w13[0].shape[0], w2[0].shape[2]
    xq = o.q_values(x)
    out = torch.zeros((T, H), dtype=F64, device=x.device)
    step = torch.zeros(T, dtype=F64, device=x.device)
    for e in range(E):
        t, j = torch.nonzero(ids == e + base, as_tuple=True)
        if t.numel() == 0:
            continue
        w, v = (o.values(codes[e], scales[e], 128) for codes, scales in (w13, w2))
        rows = xq[t].clone()
        if mistake == "the last stage of the first product lost":
            rows[:, H - 128:] = 0
        if mistake == "the last stage under the scales of the one before":
            s = w13[1][e].clone()
            s[:, -1] = s[:, -2]
            w = o.values(w13[0][e], s, 128)
        g, u = (rows @ w.T).chunk(2, dim=1)
        if mistake == "gate and up exchanged":
            g, u = u, g
        h = g * torch.sigmoid(g) * u
        hq = h if mistake == "h not quantised" else o.q_values(h)
        if mistake == "h with two bits of mantissa":
            hq = _coarse(h)
        if mistake == "eight columns of h lost":
            hq[:, 24:32] = 0
        if mistake == "the last stage of the second product lost":
            hq[:, I - 128:] = 0
        y = hq @ v.T
        if mistake == "sixteen columns of out lost":
            y[:, H - 16:] = 0
        if mistake == "the last pair of an expert lost":
            y[-1] = 0
        wt = weights[t, j].double()[:, None]
        out.index_add_(0, t, wt * y)
        cost = (hq.abs() / 8 * v.norm(dim=0)).amax(dim=1) * wt[:, 0].abs()
        step.scatter_reduce_(0, t, cost, "amax")
    return out, step


def _coarse(h):
    """h with two bits of mantissa instead of three."""
    m, e = torch.frexp(o.q_values(h))
    return torch.ldexp(torch.round(m * 8) / 8, e)


MISTAKES = ["the last stage of the first product lost", "the last stage under the scales of the one before",
            "gate and up exchanged", "h not quantised", "h with two bits of mantissa", "eight columns of h lost",
            "the last stage of the second product lost", "sixteen columns of out lost",
            "the last pair of an expert lost"]


def distance(out, x, ids, weights, w13, w2, base):
    """How far out is from the definition, in the 2-norm over all and for the worst token, each over its bound
    (within it up to 1)."""
    ref, step = forward(x, ids, weights, w13, w2, base)
    off = out.double() - ref
    if not off.isfinite().all():
        return float("inf"), float("inf")
    whole = float(off.norm() / (BOUND * ref.norm() + 1e-30))
    each = float((off.norm(dim=1) / (BOUND * ref.norm(dim=1) + 2 * step + 1e-30)).max())
    return whole, each
