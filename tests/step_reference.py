"""Plain 64-bit forms of the layer step's norm and of a cache held in 4 bits, and inputs for their tests."""
import torch

import paged_reference as ref

BLOCK_BYTES = 2304  # 16 tokens of a head: keys' codes and scales, values' codes and scales


def add_norm(x, residual, weight, eps):
    """-> (r in bf16, 64-bit y, 64-bit t = r * weight, 64-bit factor [N, 1])."""
    r = residual if x is None else (x.double() + residual.double()).to(torch.bfloat16)
    factor = (r.double().square().mean(-1, keepdim=True) + eps).rsqrt()
    t = r.double() * (1.0 if weight is None else weight.double())
    return r, t * factor, t, factor


def int8_codes(t):
    """round(127 t / T) for T the largest |t| of 128, halves to even, and T [N, H / 128]."""
    t = t.unflatten(-1, (-1, 128))
    top = t.abs().amax(-1, keepdim=True)
    return torch.where(top > 0, 127 * t / top, 0.0).round().flatten(-2).to(torch.int8), top[..., 0]


# ---------------------------------------------------------------- four bits
def quantise(x):
    """x [..., 128] bf16 -> codes [..., 128] (64-bit) and scales [..., 4] (bf16)."""
    v = x.double().unflatten(-1, (4, 32))
    s = (v.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16)
    c = torch.where(s > 0, v / s.double(), 0.0).round().clamp(-7, 7)
    return c.flatten(-2), s[..., 0]


def place():
    """For each of 128 dimensions the byte of a token's 64 that holds its code, and the bit it starts at."""
    dim = torch.arange(128)
    word = 4 * (dim % 32 // 4) + dim // 32
    return 2 * word + dim % 4 // 2, 4 * (dim % 2)


def pack_rows(codes):
    """codes [..., 128] in -8 .. 7 -> [..., 64] bytes."""
    byte, bit = place()
    n = (codes + 8).to(torch.uint8)
    low, high = (torch.argsort(byte + 64 * (bit != b)).to(codes.device)[:64] for b in (0, 4))
    return n[..., low] | n[..., high] << 4


def unpack_rows(raw):
    byte, bit = (x.to(raw.device) for x in place())
    return ((raw[..., byte].int() >> bit) & 15) - 8


class Kv4:
    """A 4-bit cache of random rows; the scales of rows nobody owns are NaN, unowned table entries out of range."""

    def __init__(self, lens, h_kv, page, dev, seed=0, spare=3, extra=1, num_pages=None, spread=0.0, codes_lo=-7):
        g = torch.Generator().manual_seed(seed)
        need = [ref.up(max(n, 0), page) for n in lens]
        self.page, self.h_kv, self.lens = page, h_kv, list(lens)
        num_pages = num_pages or sum(need) + spare
        order = torch.randperm(num_pages, generator=g).tolist()
        self.table = torch.full((len(lens), max(need, default=0) + extra), 1 << 30, dtype=torch.int32)
        self.raw = torch.full((num_pages, h_kv, page // 16, BLOCK_BYTES), 255, dtype=torch.uint8, device=dev)  # NaN scales
        self.rows = []
        for b, n in enumerate(lens):
            n = max(n, 0)
            pages = [order.pop() for _ in range(need[b])]
            self.table[b, :need[b]] = torch.tensor(pages, dtype=torch.int32)
            rows = []
            for _ in range(2):
                c = torch.randint(codes_lo, 8, (n, h_kv, 128), generator=g)
                s = (0.1 + 0.2 * torch.rand(n, h_kv, 4, generator=g)) * 10 ** (spread * torch.randn(n, h_kv, 4, generator=g))
                rows.append((c.to(dev), s.to(torch.bfloat16).to(dev)))
            self.rows.append(rows)
            self.put(b, slice(0, n), *rows)
        self.free = order
        self.table = self.table.to(dev)

    def put(self, b, at, k, v):
        pos = torch.arange(max(self.lens[b], 0))[at]
        pid = self.table[b].cpu().long()[pos // self.page].to(self.raw.device)
        off = (pos % self.page).to(self.raw.device)
        for i, (c, s) in enumerate((k, v)):
            self.part(i, "codes")[pid, :, off // 16, off % 16] = pack_rows(c)
            self.part(i, "scales")[pid, :, off // 16, off % 16] = s.contiguous().view(torch.uint8).unflatten(-1, (-1,))

    def part(self, i, what):
        """A view of the keys' (0) or values' (1) bytes, [pages, h_kv, blocks, 16, 64 or 8]."""
        at = i * BLOCK_BYTES // 2
        raw = self.raw[..., at:at + 1024] if what == "codes" else self.raw[..., at + 1024:at + 1152]
        return raw.unflatten(-1, (16, -1))

    def values(self, b):
        """Keys and values of sequence b in 64 bits, [n, h_kv, 128]."""
        return [c.double() * s.double().repeat_interleave(32, -1) for c, s in self.rows[b]]

    def hide(self, b, unseen):
        """Rows nobody sees get NaN scales; pages wholly unseen a table entry out of range."""
        n = int(unseen.sum())
        dev = self.raw.device
        bad = (torch.randint(-8, 8, (n, self.h_kv, 128), device=dev), torch.full((n, self.h_kv, 4), float("nan"),
                                                                                 dtype=torch.bfloat16, device=dev))
        self.put(b, unseen.cpu(), bad, bad)
        for i in range(ref.up(self.lens[b], self.page)):
            if unseen[i * self.page:min(self.lens[b], (i + 1) * self.page)].all():
                self.table[b, i] = -7 if i % 2 else 1 << 30


def attend(q, k, v, see, scale, k_scales=None):
    """q [h_q, 128], k and v [L, h_kv, 128] in 64 bits, see [L], k_scales [L, h_kv, 4] -> (output, sum of p |v|, largest
    p * |v|, what the scores' fp32 sums may do) in 64 bits.

    The last: a group's sum is of products n q of at most 15 |q| and its offset -8 sum(q), in fp32; two matrix instructions of
    eight products a lane's pair each, the start, the scale, the sum over groups and the unit are 8 roundings or truncations of
    at most 2^-23 of 15 sum|q| each, so a score is off by at most d = |scale| 15 2^-20 sum_w s_w sum_w|q|. A weight p changes
    by p (exp(d) - 1) at most, e for short, the output then by (sum(e |v|) + |o| sum(e)) / (1 - sum(e)).
    """
    h_q, d = q.shape
    L, h_kv, _ = k.shape
    if not bool(see.any()):
        z = torch.zeros(h_q, d, dtype=torch.float64, device=q.device)
        return z, z.clone(), z.clone(), z.clone()
    k, v = k[see].permute(1, 0, 2), v[see].permute(1, 0, 2)
    qq = q.double().view(h_kv, -1, d)
    p = torch.softmax(qq @ k.transpose(1, 2) * scale, -1)
    top = (p[..., None] * v.abs().amax(-1)[:, None, :, None]).amax(2).expand(-1, -1, d)
    out = p @ v
    slack = torch.zeros_like(out)
    if k_scales is not None:
        off = qq.abs().unflatten(-1, (4, 32)).sum(-1) @ k_scales[see].double().permute(1, 2, 0) * abs(scale) * 15 * 2.0 ** -20
        e = p * off.clamp(max=700).expm1()
        total = e.sum(-1, keepdim=True)
        slack = (e @ v.abs() + out.abs() * total) / (1 - total)
        slack = torch.where(total < 0.5, slack, torch.inf)  # scores of tens of thousands: fp32 does not settle the weights
    return tuple(x.reshape(h_q, d) for x in (out, p @ v.abs(), top, slack))


def check(got, want, size, top, slack, keys, what):
    """A probability times a value scale is rounded to fp16 once (half a step, 2^-11, of p |v|; where it is small next to
    the largest, 2^-31 of that, times a code of up to 8 against the largest value's 1 at least, for each key), the output
    to bf16 once (2^-8); 2^-12 of sum p |v| + 1e-6 stand for the approximate 2^x and the fp32 sums, slack for the scores."""
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    over = (g - want).abs() - ((2.0 ** -11 + 2.0 ** -12) * size + keys * 2.0 ** -28 * top + slack + 2.0 ** -8 * want.abs() + 1e-6)
    assert over.max() <= 0, f"{what}: {(over > 0).sum()} values out of bound, by {over.max():.3g}"
