"""Plain 64-bit forms of the operators over a paged key/value cache, and inputs for their tests."""
import torch


def up(a, b):
    return -(-a // b)


def plan(ctx, new, page, num_pages, free, count, table, n_rows):
    """moe_paged_plan by its definition, on Python lists. Returns a dict of its outputs and the status."""
    table = [list(r) for r in table]
    width = len(table[0])
    status = 0
    if not 0 <= count <= len(free):
        status, count = 7, min(max(count, 0), len(free))
    cu, needed, taken = [0], 0, 0
    seq_lens, positions, slots = [], [0] * n_rows, [-1] * n_rows
    total = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        ok = c >= 0 and n >= 0
        if not ok:
            status = max(status, 4)
        c, n = max(c, 0), max(n, 0)
        begin, total = total, total + n
        cu.append(min(total, n_rows))
        need = up(c + n, page) - up(c, page)
        if ok and (up(c + n, page) > width or total > n_rows):
            ok, status = False, 7
        if ok:
            needed += need
            if need and needed > count:
                ok, status = False, 7
        if ok:
            for k in range(need):
                table[b][up(c, page) + k] = free[count - 1 - taken - k]
            taken += need
        seq_lens.append(c + n if ok else 0)
        for i in range(min(n, n_rows - min(begin, n_rows))):
            positions[begin + i] = c + i
            if ok:
                pid = table[b][(c + i) // page]
                if 0 <= pid < num_pages:
                    slots[begin + i] = pid * page + (c + i) % page
                else:
                    status = max(status, 6)
    return dict(table=table, seq_lens=seq_lens, cu=cu, positions=positions, slots=slots, left=count - taken,
                status=status)


def norm_rope(x, weight, eps, positions, inv_freq, interleaved):
    """x [N, heads, d] -> (64-bit result, per element |a| + |b| of its rotated pair, for the tolerance)."""
    x = x.double().clone()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    size = x.abs()
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    if rot:
        angle = (positions.double()[:, None] * inv_freq.double()[None, :])[:, None, :]
        first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
        second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
        a, b = x[..., first].clone(), x[..., second].clone()
        x[..., first], x[..., second] = a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()
        size[..., first] = size[..., second] = a.abs() + b.abs()
    return x, size


def visible(pos, key, window, n_sink):
    see = (key <= pos) & (pos >= 0)
    return see & ((key > pos - window) | (key < n_sink)) if window else see


def attend(q, k, v, see, scale):
    """q [n, h_q, d], k and v [L, h_kv, d], see [n, L] -> (64-bit output, sum of p |v|), zeros where nothing is seen."""
    n, h_q, d = q.shape
    L, h_kv, _ = k.shape
    if L == 0:
        z = torch.zeros(n, h_q, d, dtype=torch.float64, device=q.device)
        return z, z.clone()
    g = h_q // h_kv
    q = q.double().view(n, h_kv, g, d).permute(1, 2, 0, 3).reshape(h_kv, g * n, d)
    unseen = ~see.any(0)  # rows nobody sees may hold anything
    k, v = k.double().clone(), v.double().clone()
    k[unseen], v[unseen] = 0, 0
    k, v = k.permute(1, 0, 2), v.permute(1, 0, 2)
    x = (q @ k.transpose(1, 2) * scale).view(h_kv, g, n, L).masked_fill(~see, -torch.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e300))
    p = x / x.sum(-1, keepdim=True).clamp(min=1e-300)
    back = lambda o: o.view(h_kv, g, n, d).permute(2, 0, 1, 3).reshape(n, h_q, d)  # noqa: E731
    p = p.view(h_kv, g * n, L)
    return back(p @ v), back(p @ v.abs())


def check(got, ref, size, what):
    """Probabilities rounded to bf16 (half a step, 2^-8 of p |v| each), the output rounded to bf16 once (2^-8 |o|),
    and 2^-12 of sum p |v| + 1e-6 for the fp32 scores, the approximate 2^x and the fp32 sums."""
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    over = (g - ref).abs() - ((2.0 ** -8 + 2.0 ** -12) * size + 2.0 ** -8 * ref.abs() + 1e-6)
    assert over.max() <= 0, f"{what}: {(over > 0).sum()} values out of bound, worst at " \
        f"{tuple(torch.unravel_index(over.argmax(), over.shape))}, by {over.max():.3g}"


class Cache:
    """A paged cache of random rows; every row no query sees is NaN, unowned table entries are out of range."""

    def __init__(self, lens, h_kv, page, dev, seed=0, spare=3, extra=1, num_pages=None, d=128):
        g = torch.Generator().manual_seed(seed)
        need = [up(max(n, 0), page) for n in lens]
        self.page, self.h_kv, self.lens = page, h_kv, list(lens)
        num_pages = num_pages or sum(need) + spare
        order = torch.randperm(num_pages, generator=g).tolist()
        self.table = torch.full((len(lens), max(need, default=0) + extra), 1 << 30, dtype=torch.int32)
        self.k = torch.full((num_pages, h_kv, page, d), float("nan"), dtype=torch.bfloat16, device=dev)
        self.v = self.k.clone()
        self.rows = []
        for b, n in enumerate(lens):
            pages = [order.pop() for _ in range(need[b])]
            self.table[b, :need[b]] = torch.tensor(pages, dtype=torch.int32)
            rows = [torch.randn(max(n, 0), h_kv, d, generator=g).to(torch.bfloat16).to(dev) for _ in range(2)]
            self.rows.append(rows)
            self.put(b, slice(0, max(n, 0)), *rows)
        self.free = order
        self.table = self.table.to(dev)

    def put(self, b, at, k, v):
        pos = torch.arange(self.lens[b])[at]
        pid = self.table[b].cpu().long()[pos // self.page].to(self.k.device)
        off = (pos % self.page).to(self.k.device)
        self.k[pid, :, off], self.v[pid, :, off] = k, v

    def hide(self, b, unseen):
        """Rows nobody sees become NaN; pages wholly unseen get a table entry out of range."""
        dev = self.k.device
        nan = torch.full((int(unseen.sum()), self.h_kv, self.k.shape[-1]), float("nan"), dtype=torch.bfloat16, device=dev)
        self.put(b, unseen.cpu(), nan, nan)
        n = self.lens[b]
        for i in range(up(n, self.page)):
            if unseen[i * self.page:min(n, (i + 1) * self.page)].all():
                self.table[b, i] = -7 if i % 2 else 1 << 30
