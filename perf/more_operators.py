"""What is measured of the layer step around the attention, and of attention over a paged cache held in 4 bits.

  norm     the residual's addition and the root-mean-square norm, its result in bf16 or
           in 8 bits with a scale for 128 dimensions                moe_add_rms_norm
  mrope    per-head norm of queries and keys with a rotation whose pairs follow several
           position axes, keys and values stored to the bf16 cache  moe_qk_norm_mrope
  store    the same norm and rotation with keys and values stored in 4 bits, and the new
           rows read back in bf16, as prompts attend to them        moe_qk_norm_rope_kv4, moe_kv4_load
  decode   one token per sequence over the 4-bit cache, sliding
           window and sinks                                         moe_gqa_kv4_decode

The 4-bit cache is [pages, h_kv, page / 16, 2304] bytes. The 2304 bytes of 16 tokens are the keys' codes (64 bytes a
token), the keys' scales (4 bf16 a token, one for 32 dimensions), then the values' codes and scales. A code c in -8 .. 7
is held as c + 8; in a token's 64 bytes the 16-bit word 4 g + w holds dimensions 32 w + 4 g .. + 3, the lowest in the
lowest 4 bits. Head counts are those of this repository's attention workloads (16/2, 32/4, 32/8, 64/4, d = 128), hidden
sizes those of its expert layers.
"""
import random

import torch

own = False

D = 128
GROUP = 128  # dimensions of one 8-bit scale
DEV = "cuda"
BLOCK = 16  # tokens of a block of the 4-bit cache
BLOCK_BYTES = 2304


# ---------------------------------------------------------------- cases
def listed():
    return [
        # in front of the experts of a decode step: one token for each of 64 requests
        dict(name="norm_decode_64", op="norm", N=64, H=4096, out="bf16"),
        # the same for a prompt batch with an odd number of tokens, the widest hidden size
        dict(name="norm_prompt_8191", op="norm", N=8191, H=7168, out="bf16"),
        # a prompt chunk whose next product takes 8 bits
        dict(name="norm_int8_2048", op="norm", N=2048, H=6144, out="int8"),
        # one new token for each of 64 requests of an image and video model
        dict(name="mrope_decode_64", op="mrope", N=64, h_q=32, h_kv=4, rot=128, page=16, norm=True, interleaved=False,
             axes=3, cycled=False),
        # a video prompt: time, height and width take turns along the pairs
        dict(name="mrope_video_8191", op="mrope", N=8191, h_q=64, h_kv=4, rot=128, page=64, norm=True,
             interleaved=False, axes=3, cycled=True),
        # the newest token of each of 64 requests
        dict(name="store_decode_64", op="store", B=64, h_q=32, h_kv=4, ctx_lo=0, ctx_hi=2048, new_lo=1, new_hi=1,
             page=16, norm=True, axes=1, lens=11),
        # prompts of very different lengths in one packed batch
        dict(name="store_prompts", op="store", B=6, h_q=32, h_kv=8, ctx_lo=0, ctx_hi=0, new_lo=1, new_hi=4095, page=64,
             norm=True, axes=1, lens=6),
        # a single user: one short sequence inside its window, where latency is all there is
        dict(name="kv4_single", op="decode", B=1, h_q=16, h_kv=2, lo=700, hi=700, page=16, window=512, n_sink=4,
             lens=3),
        # a batch on window layers: long contexts of which 1024 keys and 4 first tokens stay visible
        dict(name="kv4_window_64", op="decode", B=64, h_q=64, h_kv=4, lo=512, hi=8192, page=16, window=1024, n_sink=4,
             lens=4),
        # a large batch of short and middling requests, an odd number of them
        dict(name="kv4_ragged_255", op="decode", B=255, h_q=32, h_kv=4, lo=1, hi=4096, page=32, window=0, n_sink=0,
             lens=12),
        # a batch on full layers: all keys of up to 32 thousand tokens
        dict(name="kv4_full_16", op="decode", B=16, h_q=32, h_kv=8, lo=2048, hi=32768, page=64, window=0, n_sink=0,
             lens=5),
        # the same contexts with 16 query heads to a key/value head
        dict(name="kv4_wide_24", op="decode", B=24, h_q=64, h_kv=4, lo=2048, hi=32768, page=128, window=0, n_sink=0,
             lens=13),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm", "mrope", "store", "decode", "decode"])
    lens = rng.randrange(1 << 30)
    h_q, h_kv = rng.choice([(16, 2), (32, 4), (32, 8), (64, 4)])
    page = rng.choice([16, 32, 64, 128])
    if op == "norm":
        return dict(op=op, N=_log(rng, 1, 8191), H=rng.choice([256, 4096, 6144, 7168]),
                    out=rng.choice(["bf16", "bf16", "int8"]))
    if op == "mrope":
        return dict(op=op, N=_log(rng, 1, 8191), h_q=h_q, h_kv=h_kv, rot=rng.choice([128, 128, 64, 32]), page=page,
                    norm=rng.random() < 0.7, interleaved=rng.random() < 0.3, axes=rng.choice([2, 3, 3, 4]),
                    cycled=rng.random() < 0.5)
    if op == "store":
        B = _log(rng, 1, 64)
        new_hi = _log(rng, 1, 8191 // B)
        ctx_hi = rng.choice([0, _log(rng, 1, 2048)])
        return dict(op=op, B=B, h_q=h_q, h_kv=h_kv, ctx_lo=rng.randint(0, ctx_hi), ctx_hi=ctx_hi,
                    new_lo=rng.randint(1, new_hi), new_hi=new_hi, page=page, norm=rng.random() < 0.7,
                    axes=rng.choice([1, 1, 3]), lens=lens)
    B = _log(rng, 1, 255)
    hi = _log(rng, 1, 32768 if B <= 16 else 32768 * 16 // B)
    window = 0 if rng.random() < 0.5 else _log(rng, 1, 4096)
    return dict(op=op, B=B, h_q=h_q, h_kv=h_kv, lo=rng.randint(1, hi), hi=hi, page=page, window=window,
                n_sink=rng.choice([0, 1, 4, 130]) if window else 0, lens=lens)


# ---------------------------------------------------------------- lengths (a case's own, whatever the seed)
def _draws(case, what, lo, hi):
    r = random.Random("%d %s" % (case["lens"], what))
    return [r.randint(lo, hi) for _ in range(case["B"])]


def _lengths(case):
    """(tokens in the cache before the step, new tokens) of each sequence."""
    if case["op"] == "store":
        return _draws(case, "ctx", case["ctx_lo"], case["ctx_hi"]), _draws(case, "new", case["new_lo"], case["new_hi"])
    return [n - 1 for n in _draws(case, "len", case["lo"], case["hi"])], [1] * case["B"]


def _up(a, b):
    return -(-a // b)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=g)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _tables(g, pages_of, num_pages):
    """A block table over a random order of the pages."""
    order = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    width = max(1, max(pages_of))
    table = torch.full((len(pages_of), width), -1, dtype=torch.int32, device=DEV)
    counts = _ints(pages_of).long()
    take = torch.arange(width, device=DEV)[None, :] < counts[:, None]
    table[take] = order[:int(counts.sum())]
    return table


def _random_kv4(g, num_pages, h_kv, page):
    """A 4-bit cache of about normal values."""
    cache = torch.empty(num_pages, h_kv, page // BLOCK, BLOCK_BYTES, dtype=torch.uint8, device=DEV)
    shape = cache.shape[:3] + (BLOCK, 64)
    for at in (0, BLOCK_BYTES // 2):
        nib = [torch.randn(shape, generator=g, device=DEV).mul_(3.0).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
               for _ in range(2)]
        cache[..., at:at + 1024] = (nib[0] | (nib[1] << 4)).flatten(-2)
        scales = torch.rand(cache.shape[:3] + (BLOCK * 4,), generator=g, device=DEV).mul_(0.2).add_(0.25)
        cache[..., at + 1024:at + 1152] = scales.to(torch.bfloat16).view(torch.uint8)
    return cache


def _rope_inputs(g, case, N):
    rot, axes = case.get("rot", D), case["axes"]
    s = dict(qkv=_normal(g, N, (case["h_q"] + 2 * case["h_kv"]) * D), eps=1e-6,
             q_weight=1 + 0.1 * _normal(g, D) if case["norm"] else None,
             k_weight=1 + 0.1 * _normal(g, D) if case["norm"] else None,
             inv_freq=(1e6 ** (-torch.arange(0, rot, 2, device=DEV).double() / rot)).float(),
             positions=torch.randint(0, 131072, (axes, N), generator=g, device=DEV, dtype=torch.int32),
             q_out=torch.empty(N, case["h_q"], D, dtype=torch.bfloat16, device=DEV), pair_axis=None)
    if axes > 1:
        pair = torch.arange(rot // 2, device=DEV)
        # the axes' pairs one axis after the other (the first with the fewest), or in turns
        s["pair_axis"] = (pair % axes if case.get("cycled") else (pair * axes + rot // 8).div(rot // 2, rounding_mode="floor")
                          .clamp(max=axes - 1)).to(torch.int32)
    return s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case, op=op)
    if op == "norm":
        N, H = case["N"], case["H"]
        bf16 = case["out"] == "bf16"
        empty = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
        s.update(x=_normal(g, N, H), residual=4 * _normal(g, N, H), weight=1 + 0.1 * _normal(g, H), eps=1e-6,
                 residual_out=empty(N, H, dtype=torch.bfloat16), y=empty(N, H, dtype=torch.bfloat16) if bf16 else None,
                 q=None if bf16 else empty(N, H, dtype=torch.int8),
                 scales=None if bf16 else empty(N, H // GROUP, dtype=torch.float32))
        return s
    page, h_kv = case["page"], case["h_kv"]
    if op == "mrope":
        N = case["N"]
        num_pages = _up(N, page) + 3
        s.update(_rope_inputs(g, case, N))
        s.update(slots=torch.randperm(num_pages * page, generator=g, device=DEV)[:N].to(torch.int32),
                 k_cache=_normal(g, num_pages, h_kv, page, D), v_cache=_normal(g, num_pages, h_kv, page, D))
        return s
    ctx, new = _lengths(case)
    lens = [c + n for c, n in zip(ctx, new)]
    pages_of = [_up(n, page) for n in lens]
    num_pages = sum(pages_of) + 5
    table = _tables(g, pages_of, num_pages)
    s.update(cache=_random_kv4(g, num_pages, h_kv, page), table=table, seq_lens=_ints(lens))
    if op == "store":
        N = sum(new)
        s.update(_rope_inputs(g, case, N))
        seq = torch.repeat_interleave(torch.arange(case["B"], device=DEV), _ints(new).long())
        begin = torch.cumsum(_ints(new).long(), 0) - _ints(new)
        pos = _ints(ctx).long()[seq] + torch.arange(N, device=DEV) - begin[seq]
        wide = _tables(g, pages_of, num_pages)
        s.update(ctx=_ints(ctx), seq=seq, pos=pos, wide_table=wide,
                 slots=(table[seq, pos // page].long() * page + pos % page).to(torch.int32),
                 k_wide=_normal(g, num_pages, h_kv, page, D), v_wide=_normal(g, num_pages, h_kv, page, D))
    else:
        s.update(q=_normal(g, case["B"], case["h_q"], D), scale=D ** -0.5, max_len=max(lens),
                 out=torch.empty(case["B"], case["h_q"], D, dtype=torch.bfloat16, device=DEV))
    if own:
        import routed_expert_ffn_softmax_gb300 as moe
        s["ws"] = moe.alloc_paged_workspace(case["B"], case["B"], case["h_q"], h_kv, D, device=DEV)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    return {"norm": _plain_norm, "mrope": _plain_mrope, "store": _plain_store, "decode": _plain_decode}[s["op"]](s)


def _run_own(s):
    import routed_expert_ffn_softmax_gb300 as moe
    op, case = s["op"], s["case"]
    if op == "norm":
        moe.moe_add_rms_norm(s["x"], s["residual"], s["weight"], s["eps"], s["residual_out"], s["y"], s["q"],
                             s["scales"])
        if s["y"] is not None:
            return [s["residual_out"], s["y"]]
        return [s["residual_out"], _int8_values(s["q"], s["scales"])]
    if op == "mrope":
        moe.moe_qk_norm_mrope(s["qkv"], s["q_weight"], s["k_weight"], s["eps"], s["inv_freq"], s["pair_axis"],
                              s["positions"], s["slots"], s["q_out"], s["k_cache"], s["v_cache"],
                              interleaved=case["interleaved"])
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    if op == "store":
        moe.moe_qk_norm_rope_kv4(s["qkv"], s["q_weight"], s["k_weight"], s["eps"], s["inv_freq"], s["pair_axis"],
                                 s["positions"], s["slots"], s["q_out"], s["cache"])
        moe.moe_kv4_load(s["cache"], s["table"], s["ctx"], s["seq_lens"], s["k_wide"], s["v_wide"], s["wide_table"],
                         s["ws"])
        return [s["q_out"], s["k_wide"], s["v_wide"]]
    moe.moe_gqa_kv4_decode(s["q"], s["cache"], s["table"], s["seq_lens"], s["scale"], s["out"], s["ws"],
                           window=case["window"], n_sink=case["n_sink"])
    return s["out"]


def _int8_values(q, scales):
    N, H = q.shape
    return (q.view(N, -1, GROUP) * scales[:, :, None]).view(N, H)


# ---------------------------------------------------------------- plain forms
def _plain_norm(s):
    r = (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    t = r.float()
    factor = torch.rsqrt((t * t).mean(-1, keepdim=True) + s["eps"])
    t = t * s["weight"].float()  # exact: two factors of 8 bits
    if s["y"] is not None:
        return [r, (t * factor).to(torch.bfloat16)]
    N, H = t.shape
    t = t.view(N, -1, GROUP)
    top = t.abs().amax(-1, keepdim=True)
    # the codes in 64 bits, where no quotient next to a half is rounded onto it
    codes = (t.double() * 127 / torch.where(top == 0, 1.0, top).double()).round().to(torch.int8)
    scales = torch.where(top == 0, 1.0, top * factor[:, :, None] / 127)
    return [r, _int8_values(codes.view(N, H), scales[:, :, 0])]


def _norm_rope(x, weight, eps, cos, sin, rot, interleaved):
    """x [N, heads, D] in 32 bits."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.to(x.dtype)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([lo, hi], -1).flatten(-2) if interleaved else torch.cat([lo, hi], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _pair_positions(s):
    """[N, rot / 2]: the position that each pair follows."""
    if s["pair_axis"] is None:
        return s["positions"][0][:, None]
    return s["positions"][s["pair_axis"].long()].t()


def _plain_heads(s):
    """Queries, keys and values after norm and rotation, in bf16."""
    case = s["case"]
    h_q, h_kv, rot, turns = case["h_q"], case["h_kv"], case.get("rot", D), case.get("interleaved", False)
    angle = _pair_positions(s).double() * s["inv_freq"].double()[None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    x = s["qkv"].view(-1, h_q + 2 * h_kv, D).float()
    q = _norm_rope(x[:, :h_q], s["q_weight"], s["eps"], cos, sin, rot, turns)
    k = _norm_rope(x[:, h_q:h_q + h_kv], s["k_weight"], s["eps"], cos, sin, rot, turns)
    return q.to(torch.bfloat16), k.to(torch.bfloat16), x[:, h_q + h_kv:].to(torch.bfloat16)


def _plain_mrope(s):
    page, slots = s["case"]["page"], s["slots"].long()
    q, k, v = _plain_heads(s)
    s["k_cache"][slots // page, :, slots % page] = k
    s["v_cache"][slots // page, :, slots % page] = v
    return [q, s["k_cache"], s["v_cache"]]


def _to_4_bits(x):
    """x [..., D] bf16 -> codes [..., 4, 32] and scales [..., 4, 1], both in 32 bits: code = round(x / scale)."""
    x = x.float().unflatten(-1, (4, 32))
    scale = (x.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16).float()
    codes = (x.double() / torch.where(scale == 0, 1.0, scale).double()).round().clamp(-7, 7)
    return codes.float(), scale


def _plain_store(s):
    page = s["case"]["page"]
    q, k, v = _plain_heads(s)
    to = s["wide_table"][s["seq"], s["pos"] // page].long(), s["pos"] % page
    for heads, wide in ((k, s["k_wide"]), (v, s["v_wide"])):
        codes, scale = _to_4_bits(heads)
        wide[to[0], :, to[1]] = (codes * scale).flatten(-2).to(torch.bfloat16)
    return [q, s["k_wide"], s["v_wide"]]


def _values(blocks, at, dtype):
    """[..., blocks, BLOCK_BYTES] -> [..., blocks * BLOCK, D]: the keys (at = 0) or values (at = 1152) of 4-bit blocks."""
    codes = blocks[..., at:at + 1024].unflatten(-1, (BLOCK, 8, 4, 2))  # token, g, w, byte
    codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).transpose(-2, -3)  # token, w, g, 4 dimensions
    codes = codes.flatten(-2).to(dtype) - 8
    scales = blocks[..., at + 1024:at + 1152].contiguous().view(torch.bfloat16).unflatten(-1, (BLOCK, 4))
    return (codes * scales[..., None].to(dtype)).flatten(-2).flatten(-3, -2)


def _keys(s, at, length):
    """[B, h_kv, length, D] in 32 bits, out of the pages."""
    pages = _up(length, s["case"]["page"])
    got = s["cache"][s["table"][:, :pages].clamp(min=0).long()].transpose(1, 2)
    return _values(got.flatten(2, 3), at, torch.float32)[:, :, :length]


def _plain_decode(s):
    case = s["case"]
    k, v = _keys(s, 0, s["max_len"]), _keys(s, 1152, s["max_len"])
    q = s["q"].float().view(case["B"], case["h_kv"], -1, D)
    pos = s["seq_lens"].long()[:, None, None, None] - 1
    key = torch.arange(s["max_len"], device=DEV)
    see = key <= pos
    if case["window"]:
        see = see & ((key > pos - case["window"]) | (key < case["n_sink"]))
    x = (q @ k.transpose(-1, -2) * s["scale"]).masked_fill(~see, -torch.inf)
    e = (x - x.amax(-1, keepdim=True)).exp()
    return (e @ v / e.sum(-1, keepdim=True)).to(torch.bfloat16).reshape(case["B"], case["h_q"], D)


# ---------------------------------------------------------------- the least work of a pass
def _seen(length, window, n_sink):
    """Keys the newest of `length` tokens sees."""
    if not window or length <= window:
        return length
    return window + min(n_sink, length - window)


def work(case):
    op = case["op"]
    if op == "norm":
        N, H = case["N"], case["H"]
        bf16 = case["out"] == "bf16"
        # both inputs, the sum, the weight; the result in bf16, or codes and scales
        return dict(bytes=N * H * (6 + (2 if bf16 else 1)) + 2 * H + (0 if bf16 else 4 * N * H // GROUP),
                    flops=N * H * (5 if bf16 else 8))
    h_q, h_kv = case["h_q"], case["h_kv"]
    if op in ("mrope", "store"):
        N = case["N"] if op == "mrope" else sum(_lengths(case)[1])
        rot, axes = case.get("rot", D), case["axes"]
        flops = N * (h_q + h_kv) * (3 * rot + (4 * D if case["norm"] else 0))
        small = 4 * N * (axes + 1) + 4 * rot
        if op == "mrope":
            return dict(bytes=2 * 2 * N * (h_q + 2 * h_kv) * D + small, flops=flops)
        # queries in and out, keys and values in, their 4 bits out and in again, their bf16 out
        return dict(bytes=N * D * (4 * h_q + 8 * h_kv) + 2 * N * h_kv * 2 * 72 + small,
                    flops=flops + 6 * N * h_kv * D)
    ctx, _ = _lengths(case)
    keys = sum(_seen(c + 1, case["window"], case["n_sink"]) for c in ctx)
    return dict(bytes=2 * 2 * case["B"] * h_q * D + keys * h_kv * 2 * 72, flops=4 * D * h_q * keys)


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "mrope": _exact_mrope, "store": _exact_store, "decode": _exact_decode}[case["op"]](case, s)


def _exact_norm(case, s):
    N, H = case["N"], case["H"]
    out = [torch.empty(N, H, dtype=torch.float64, device=DEV) for _ in range(2)]
    for i in range(0, N, 1024):
        rows = slice(i, i + 1024)
        r = s["x"][rows].double().add_(s["residual"][rows]).to(torch.bfloat16).double()
        y = r * s["weight"].double() / (r.square().sum(-1, keepdim=True) / H + s["eps"]).sqrt()
        if case["out"] == "int8":
            y = y.unflatten(-1, (-1, GROUP))
            # the ratio to the group's largest does not depend on the norm
            t = (r * s["weight"].double()).unflatten(-1, (-1, GROUP))
            top = t.abs().amax(-1, keepdim=True)
            codes = torch.where(top > 0, t * 127 / top, 0.0).round()
            y = (codes * (y.abs().amax(-1, keepdim=True) / 127)).flatten(-2)
        out[0][rows], out[1][rows] = r, y
    return out


def _exact_heads(case, s):
    h_q, h_kv, rot, turns = case["h_q"], case["h_kv"], case.get("rot", D), case.get("interleaved", False)
    x = s["qkv"].double().view(-1, h_q + 2 * h_kv, D)
    parts = [x[:, :h_q].clone(), x[:, h_q:h_q + h_kv].clone()]
    theta = torch.empty(x.shape[0], rot // 2, dtype=torch.float64, device=DEV)
    for i in range(rot // 2):
        axis = 0 if s["pair_axis"] is None else int(s["pair_axis"][i])
        theta[:, i] = s["positions"][axis].double() * s["inv_freq"][i].double()
    turn = torch.polar(torch.ones_like(theta), theta)[:, None, :]  # e^(i theta)
    first = slice(0, rot, 2) if turns else slice(0, rot // 2)
    second = slice(1, rot, 2) if turns else slice(rot // 2, rot)
    for part, w in zip(parts, (s["q_weight"], s["k_weight"])):
        if w is not None:
            part.div_((part.square().sum(-1, keepdim=True) / D + s["eps"]).sqrt()).mul_(w.double())
        z = torch.complex(part[..., first], part[..., second]) * turn
        part[..., first], part[..., second] = z.real.clone(), z.imag.clone()
    return parts[0], parts[1], x[:, h_q + h_kv:]


def _place(wide, page, pid, off, rows):
    out = wide.double()
    flat = out.transpose(1, 2).reshape(-1, wide.shape[1], D)
    flat[pid * page + off] = rows
    return flat.view(-1, page, wide.shape[1], D).transpose(1, 2).contiguous()


def _exact_mrope(case, s):
    q, k, v = _exact_heads(case, s)
    pid, off = s["slots"].long() // case["page"], s["slots"].long() % case["page"]
    return [q] + [_place(c, case["page"], pid, off, rows) for c, rows in ((s["k_cache"], k), (s["v_cache"], v))]


def _exact_store(case, s):
    q, k, v = _exact_heads(case, s)
    pid, off = s["wide_table"][s["seq"], s["pos"] // case["page"]].long(), s["pos"] % case["page"]
    out = [q]
    for wide, rows in ((s["k_wide"], k), (s["v_wide"], v)):
        rows = rows.to(torch.bfloat16).double()  # what is held in 4 bits are the values of the bf16 cache
        for w in range(4):
            part = rows[..., 32 * w:32 * w + 32]
            unit = (part.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16).double()
            part.copy_(torch.where(unit > 0, part / unit, 0.0).round().clamp(-7, 7) * unit)
        out.append(_place(wide, case["page"], pid, off, rows))
    return out


def _exact_decode(case, s):
    h_q, h_kv, page = case["h_q"], case["h_kv"], case["page"]
    group = h_q // h_kv
    ctx, _ = _lengths(case)
    table = s["table"].cpu().tolist()
    out = torch.zeros(case["B"], h_q, D, dtype=torch.float64, device=DEV)
    # where each dimension's code stands in a token's 64 bytes
    dim = torch.arange(D, device=DEV)
    w, g, i = dim // 32, dim % 32 // 4, dim % 4
    byte, shift = 2 * (4 * g + w) + i // 2, 4 * (i % 2)

    def rows(blocks, at):
        code = (blocks[:, at:at + 1024].reshape(-1, 64)[:, byte].int() >> shift & 15) - 8
        unit = blocks[:, at + 1024:at + 1152].contiguous().view(torch.bfloat16).reshape(-1, 4).double()
        return code.double() * unit[:, w]

    for b, c in enumerate(ctx):
        length = c + 1
        first = max(0, length - case["window"]) if case["window"] else 0
        keep = torch.arange(length, device=DEV)
        keep = keep[(keep >= first) | (keep < case["n_sink"])]
        pages = table[b][:_up(length, page)]
        for j in range(h_kv):
            blocks = s["cache"][pages, j].reshape(-1, BLOCK_BYTES)
            k, v = rows(blocks, 0)[keep], rows(blocks, 1152)[keep]
            q = s["q"][b, j * group:(j + 1) * group].double()
            out[b, j * group:(j + 1) * group] = torch.softmax(q @ k.T * s["scale"], -1) @ v
    return out
