"""Plain CPU forms of the 8-bit operators for the tests, and their bounds.

* e4m3 codes and fp32 scales come from the formulas with every operation in
  fp32 (torch on the CPU rounds each one to nearest), so the quantisers are
  compared bit for bit.
* A product is compared with the float64 sum of what codes and scales stand
  for.  A group's 128 products are exact in fp32 (4-bit significands); adding
  them on the tensor core and the groups in fp32 takes fewer than
  128 + 2 groups roundings of partial sums, each at most S = sum |x w| of the
  whole row, by at most 2^-23 (truncation counted), and the scales' product,
  the parts' sums and the bias a few more: |err| <= (128 + 2 G + 8) 2^-23 S.
  (A K block's own sum is bounded by its own S; the bound is generous by that.)
  A bf16 output adds half a step, 2^-8 |y|.
* Rounding v to e4m3 with scale s moves it by at most 2^-4 |v|, or half of
  the subnormal step 2^-9 s.
"""

import torch

FP8 = torch.float8_e4m3fn
G = 128


def groups(k):
    return -(-k // G)


def _scale(amax):
    least = torch.full_like(amax, 2.0 ** -100)
    a = torch.where(torch.isnan(amax), amax, torch.maximum(amax, least))
    return a / torch.full_like(amax, 448.0)


def _e4m3(q):
    """float32 -> e4m3 codes; past the range saturates as the GPU's conversion does."""
    q = torch.where(q.isfinite() | q.isnan(), q, torch.copysign(torch.full_like(q, 448.0), q))
    return q.to(FP8)


def quantise_rows(x):
    """(codes [n, k], scales [groups, n]) of a CPU tensor."""
    x = x.float()
    n, k = x.shape
    v = torch.nn.functional.pad(x, (0, -k % G)).reshape(n, groups(k), G)
    s = _scale(v.abs().amax(-1))
    q = (v / s[..., None]).reshape(n, -1)[:, :k]
    return _e4m3(q), s.t().contiguous()


def quantise_weight(w, gated=False):
    if gated:
        half = w.shape[0] // 2
        a, b = quantise_weight(w[:half]), quantise_weight(w[half:])
        return (torch.cat([a[0].view(torch.uint8), b[0].view(torch.uint8)]).view(FP8), torch.cat([a[1], b[1]]))
    w = w.float()
    out, k = w.shape
    v = torch.nn.functional.pad(w, (0, -k % G, 0, -out % G)).reshape(groups(out), G, groups(k), G)
    s = _scale(v.abs().amax((1, 3)))
    q = (v / s[:, None, :, None]).reshape(groups(out) * G, -1)[:out, :k]
    return _e4m3(q.contiguous()), s.contiguous()


def rows64(codes, scales):
    """float64 values of rows."""
    k = codes.shape[1]
    return codes.cpu().to(torch.float64) * scales.cpu().double().t().repeat_interleave(G, 1)[:, :k]


def weight64(codes, scales):
    out, k = codes.shape
    s = scales.cpu().double().repeat_interleave(G, 0)[:out].repeat_interleave(G, 1)[:, :k]
    return codes.cpu().to(torch.float64) * s


def halves64(codes, scales):
    """float64 gate and up weights of a gated block."""
    half, blocks = codes.shape[0] // 2, scales.shape[0] // 2
    return weight64(codes[:half], scales[:blocks]), weight64(codes[half:], scales[blocks:])


def product(xs, ws, bias=None):
    """(y, bound) of sum_r x_r w_r^T in float64: xs, ws lists of float64 matrices."""
    y = sum(x @ w.t() for x, w in zip(xs, ws))
    s = sum(x.abs() @ w.abs().t() for x, w in zip(xs, ws))
    g = sum(groups(x.shape[1]) for x in xs)
    if bias is not None:
        y, s = y + bias.double().cpu(), s + bias.double().cpu().abs()
    return y, (128 + 2 * g + 8) * 2.0 ** -23 * s + 1e-37


def act64(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g ** 3)))


def gated(x, gate, up, act):
    """(act(gate) * up, bound) in float64."""
    a, ea = product([x], [gate])
    u, eu = product([x], [up])
    v = act64(a, act) * u
    # |act'| <= 1.13 for both; the fast exponential, divide and tanh: within 2^-20 of act's value or of |g|'s
    e = 1.13 * ea * u.abs() + act64(a, act).abs() * eu + 1.13 * ea * eu + 2.0 ** -20 * a.abs() * u.abs()
    return v, e + 1e-37


def held(v, e, scales):
    """Bound on what codes with `scales` [groups, n] may be off a value known to e: half an e4m3 step of the value
    (2^-4 of it, or half the subnormal step), the value's own bound, and twice fp32's rounding of scale and quotient."""
    s = scales.cpu().double().t().repeat_interleave(G, 1)[:, :v.shape[1]]
    return e * (1 + 2.0 ** -4) + torch.maximum(2.0 ** -4 * (v.abs() + e), 2.0 ** -10 * s) + 2.0 ** -22 * v.abs()
