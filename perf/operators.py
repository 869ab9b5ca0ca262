"""What is measured of the serving path over a paged key/value cache: one decode or prompt step in front of the
routed experts, operator by operator.

  plan     block tables and slot maps from request lengths      moe_paged_plan
  qk       per-head norm of queries and keys with the rotation,
           keys and values stored to the cache                    moe_qk_norm_rope
  decode   one token per sequence, sliding window and sinks      moe_gqa_paged_decode
  prompt   many tokens per sequence, the same masks              moe_gqa_paged_prefill
  prefix   one token per sequence behind a prefix all share      moe_gqa_prefix_decode

The cache is [pages, h_kv, page, d]; a sequence's keys are found through its row of the block table. Head counts are
those of this repository's attention workloads (16/2, 32/4, 32/8, 64/4, d = 128).
"""
import random

import torch

own = False

D = 128
DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the step before every decode step of a serving loop: one new token for each of 64 requests
        dict(name="plan_decode_64", op="plan", B=64, ctx_lo=512, ctx_hi=8192, new_lo=1, new_hi=1, page=16, lens=1),
        # prompts being admitted beside running requests: many sequences, about 66 thousand new tokens
        dict(name="plan_admit_1000", op="plan", B=1000, ctx_lo=0, ctx_hi=4096, new_lo=1, new_hi=131, page=16, lens=2),
        # one new token for each of 64 requests
        dict(name="qk_decode_64", op="qk", N=64, h_q=32, h_kv=4, rot=128, page=16, norm=True, interleaved=False),
        # a prompt batch with an odd number of tokens, the widest head layout
        dict(name="qk_prompt_8191", op="qk", N=8191, h_q=64, h_kv=4, rot=128, page=64, norm=True, interleaved=False),
        # a single user: one short sequence inside its window, where latency is all there is
        dict(name="decode_single", op="decode", B=1, h_q=16, h_kv=2, lo=700, hi=700, page=16, window=512, n_sink=4,
             lens=3),
        # a batch on window layers: long contexts of which 1024 keys and 4 first tokens stay visible
        dict(name="decode_window_64", op="decode", B=64, h_q=64, h_kv=4, lo=512, hi=8192, page=16, window=1024,
             n_sink=4, lens=4),
        # a batch on full layers: all keys of up to 32 thousand tokens
        dict(name="decode_full_16", op="decode", B=16, h_q=32, h_kv=8, lo=2048, hi=32768, page=64, window=0, n_sink=0,
             lens=5),
        # prompts of very different lengths in one packed batch, full causal attention
        dict(name="prompt_ragged", op="prompt", B=6, h_q=32, h_kv=8, ctx_lo=0, ctx_hi=0, new_lo=1, new_hi=4095,
             page=64, window=0, n_sink=0, lens=6),
        # one long prompt on a window layer
        dict(name="prompt_window_16k", op="prompt", B=1, h_q=16, h_kv=2, ctx_lo=0, ctx_hi=0, new_lo=16384,
             new_hi=16384, page=128, window=4096, n_sink=4, lens=7),
        # several tokens per request behind long contexts (drafted tokens to verify, chunks of prompts)
        dict(name="prompt_chunk_8", op="prompt", B=8, h_q=32, h_kv=4, ctx_lo=1000, ctx_hi=16000, new_lo=1, new_hi=65,
             page=16, window=0, n_sink=0, lens=8),
        # requests behind one system prompt of 8192 tokens
        dict(name="prefix_64", op="prefix", B=64, h_q=32, h_kv=4, prefix=8192, lo=1, hi=1024, page=16, lens=9),
        # many samples of one document of 32 thousand tokens, an odd number of them
        dict(name="prefix_255", op="prefix", B=255, h_q=64, h_kv=4, prefix=32768, lo=0, hi=512, page=64, lens=10),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["plan", "qk", "decode", "prompt", "prefix"])
    lens = rng.randrange(1 << 30)
    h_q, h_kv = rng.choice([(16, 2), (32, 4), (32, 8), (64, 4)])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _log(rng, 1, 1000)
        new_hi = _log(rng, 1, 131)
        ctx_hi = _log(rng, 1, 8192)
        return dict(op=op, B=B, ctx_lo=rng.randint(0, ctx_hi), ctx_hi=ctx_hi, new_lo=rng.randint(1, new_hi),
                    new_hi=new_hi, page=page, lens=lens)
    if op == "qk":
        return dict(op=op, N=_log(rng, 1, 8191), h_q=h_q, h_kv=h_kv, rot=rng.choice([128, 128, 64, 32]), page=page,
                    norm=rng.random() < 0.7, interleaved=rng.random() < 0.3)
    if op == "decode":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, 32768 * 16 // max(16, B) if B > 16 else 32768)
        window = 0 if rng.random() < 0.3 else _log(rng, 1, 4096)
        return dict(op=op, B=B, h_q=h_q, h_kv=h_kv, lo=rng.randint(1, hi), hi=hi, page=page, window=window,
                    n_sink=rng.choice([0, 1, 4, 130]) if window else 0, lens=lens)
    if op == "prompt":
        B = _log(rng, 1, 8)
        new_hi = _log(rng, 1, 4095 // B)
        ctx_hi = rng.choice([0, _log(rng, 1, 8000)])
        window = 0 if rng.random() < 0.5 else _log(rng, 1, 4096)
        case = dict(op=op, B=B, h_q=h_q, h_kv=h_kv, ctx_lo=rng.randint(0, ctx_hi), ctx_hi=ctx_hi,
                    new_lo=rng.randint(1, new_hi), new_hi=new_hi, page=page, window=window,
                    n_sink=rng.choice([0, 1, 4, 130]) if window else 0, lens=lens)
        while work(case)["flops"] > 4e11:  # no more than the largest listed prompt
            case["new_hi"] = case["new_hi"] // 2 + 1
            case["new_lo"] = min(case["new_lo"], case["new_hi"])
        return case
    hi = _log(rng, 1, 512)
    return dict(op=op, B=_log(rng, 1, 255), h_q=h_q, h_kv=h_kv, prefix=_log(rng, 16, 32768), lo=rng.randint(0, hi),
                hi=hi, page=page, lens=lens)


# ---------------------------------------------------------------- lengths (a case's own, whatever the seed)
def _draws(case, what, lo, hi):
    r = random.Random("%d %s" % (case["lens"], what))
    return [r.randint(lo, hi) for _ in range(case["B"])]


def _lengths(case):
    """(tokens in the cache before the step, new tokens) of each sequence."""
    if case["op"] in ("plan", "prompt"):
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
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        flat[i:i + step].normal_(generator=g)
    return out


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _tables(g, pages_of, num_pages):
    """A block table over a random order of the pages, and the order's rest."""
    order = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    width = max(1, max(pages_of))
    table = torch.full((len(pages_of), width), -1, dtype=torch.int32, device=DEV)
    counts = _ints(pages_of).long()
    take = torch.arange(width, device=DEV)[None, :] < counts[:, None]
    table[take] = order[:int(counts.sum())]
    return table, order[int(counts.sum()):].contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op, page = case["op"], case["page"]
    s = dict(case=case, op=op)
    if op == "plan":
        ctx, new = _lengths(case)
        owned = [_up(c, page) for c in ctx]
        need = [_up(c + n, page) for c, n in zip(ctx, new)]
        spare = 64
        num_pages = sum(need) + spare
        table, free = _tables(g, owned, num_pages)
        width = max(need) + 8
        block_table = torch.full((case["B"], width), -1, dtype=torch.int32, device=DEV)
        block_table[:, :table.shape[1]] = table[:, :width]
        cap = _up(sum(new), 64) * 64
        s.update(ctx=_ints(ctx), new=_ints(new), page=page, num_pages=num_pages, free=free,
                 free_count=_ints([free.numel()]), table=block_table, seq_lens=_ints([0] * case["B"]),
                 cu=_ints([0] * (case["B"] + 1)), positions=torch.zeros(cap, dtype=torch.int32, device=DEV),
                 slots=torch.zeros(cap, dtype=torch.int32, device=DEV), left=_ints([0]))
    elif op == "qk":
        N, h_q, h_kv = case["N"], case["h_q"], case["h_kv"]
        num_pages = _up(N, page) + 3
        s.update(qkv=_normal(g, N, (h_q + 2 * h_kv) * D), eps=1e-6,
                 q_weight=1 + 0.1 * _normal(g, D) if case["norm"] else None,
                 k_weight=1 + 0.1 * _normal(g, D) if case["norm"] else None,
                 inv_freq=1e6 ** (-torch.arange(0, case["rot"], 2, device=DEV).double() / case["rot"]),
                 positions=torch.randint(0, 131072, (N,), generator=g, device=DEV, dtype=torch.int32),
                 slots=torch.randperm(num_pages * page, generator=g, device=DEV)[:N].to(torch.int32),
                 q_out=torch.empty(N, h_q, D, dtype=torch.bfloat16, device=DEV),
                 k_cache=_normal(g, num_pages, h_kv, page, D), v_cache=_normal(g, num_pages, h_kv, page, D))
        s["inv_freq"] = s["inv_freq"].float()
    else:
        ctx, new = _lengths(case)
        lens = [c + n for c, n in zip(ctx, new)]
        pages_of = [_up(n, page) for n in lens]
        shared = _up(case.get("prefix", 0), page)
        num_pages = sum(pages_of) + shared + 5
        table, rest = _tables(g, pages_of, num_pages)
        N = sum(new)
        s.update(q=_normal(g, N, case["h_q"], D), k_cache=_normal(g, num_pages, case["h_kv"], page, D),
                 v_cache=_normal(g, num_pages, case["h_kv"], page, D), table=table, seq_lens=_ints(lens),
                 scale=D ** -0.5, out=torch.empty(N, case["h_q"], D, dtype=torch.bfloat16, device=DEV),
                 max_len=max(lens), max_new=max(new))
        if op == "prompt":
            cu = [0]
            for n in new:
                cu.append(cu[-1] + n)
            s["cu"] = _ints(cu)
        if op == "prefix":
            s.update(prefix_table=rest[:shared].contiguous(), prefix=case["prefix"])
    if own:
        import routed_expert_ffn_softmax_gb300 as moe
        if op == "plan":
            s["ws"] = moe.alloc_paged_workspace(device=DEV)
        elif op != "qk":
            s["ws"] = moe.alloc_paged_workspace(s["q"].shape[0], case["B"], case["h_q"], case["h_kv"], D,
                                                case.get("prefix", 0), device=DEV)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    return {"plan": _plain_plan, "qk": _plain_qk, "decode": _plain_decode, "prompt": _plain_prompt,
            "prefix": _plain_prefix}[s["op"]](s)


def _run_own(s):
    import routed_expert_ffn_softmax_gb300 as moe
    op, case = s["op"], s["case"]
    if op == "plan":
        moe.moe_paged_plan(s["ctx"], s["new"], s["page"], s["num_pages"], s["free"], s["free_count"], s["table"],
                           s["seq_lens"], s["cu"], s["positions"], s["slots"], s["left"], s["ws"])
        return [s[k] for k in ("table", "seq_lens", "cu", "positions", "slots", "left")]
    if op == "qk":
        moe.moe_qk_norm_rope(s["qkv"], s["q_weight"], s["k_weight"], s["eps"], s["inv_freq"], s["positions"],
                             s["slots"], s["q_out"], s["k_cache"], s["v_cache"], interleaved=case["interleaved"])
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    if op == "decode":
        moe.moe_gqa_paged_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"], s["scale"], s["out"],
                                 s["ws"], window=case["window"], n_sink=case["n_sink"])
    elif op == "prompt":
        moe.moe_gqa_paged_prefill(s["q"], s["cu"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"], s["scale"],
                                  s["out"], s["ws"], window=case["window"], n_sink=case["n_sink"])
    else:
        moe.moe_gqa_prefix_decode(s["q"], s["prefix_table"], s["prefix"], s["k_cache"], s["v_cache"], s["table"],
                                  s["seq_lens"], s["scale"], s["out"], s["ws"])
    return s["out"]


# ---------------------------------------------------------------- plain forms
def _plain_plan(s):
    page, table, free = s["page"], s["table"], s["free"]
    ctx, new = s["ctx"].long(), s["new"].long()
    B, width = table.shape
    cap = s["positions"].shape[0]
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), new.cumsum(0)])
    owned = (ctx + page - 1) // page
    need = (ctx + new + page - 1) // page - owned
    good = (owned + need <= width) & (cu[1:] <= cap)
    need = torch.where(good, need, 0)
    last = need.cumsum(0)
    count = s["free_count"].long()
    fits = good & ((need == 0) | (last <= count))
    seq_lens = torch.where(fits, ctx + new, 0)
    # new pages come off the end of the free list, in order of (sequence, page)
    col = torch.arange(width, device=DEV)[None, :]
    fresh = (col >= owned[:, None]) & (col < (owned + need)[:, None]) & fits[:, None]
    nth = (last - need)[:, None] + col - owned[:, None]
    taken = free[(count - 1 - nth).clamp(0, max(0, free.numel() - 1))] if free.numel() else torch.zeros_like(table)
    table = torch.where(fresh, taken, table)
    tok = torch.arange(cap, device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), tok, right=True).clamp(max=B - 1)
    pos = ctx[seq] + tok - cu[seq]
    real = tok < cu[-1]
    slot = table[seq, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    slots = torch.where(real & fits[seq], slot, -1)
    positions = torch.where(real, pos, 0)
    left = count - torch.where(fits, need, 0).sum()
    return [t.to(torch.int32) for t in (table, seq_lens, cu.clamp(max=cap), positions, slots, left)]


def _norm_rope(x, weight, eps, cos, sin, rot, interleaved):
    """x [N, heads, D] in 32 bits (or 64, for exact())."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.to(x.dtype)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([lo, hi], -1).flatten(-2) if interleaved else torch.cat([lo, hi], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_qk(s):
    case = s["case"]
    h_q, h_kv, page = case["h_q"], case["h_kv"], case["page"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    x = s["qkv"].view(-1, h_q + 2 * h_kv, D).float()
    q = _norm_rope(x[:, :h_q], s["q_weight"], s["eps"], cos, sin, case["rot"], case["interleaved"])
    k = _norm_rope(x[:, h_q:h_q + h_kv], s["k_weight"], s["eps"], cos, sin, case["rot"], case["interleaved"])
    slots = s["slots"].long()
    s["k_cache"][slots // page, :, slots % page] = k.to(torch.bfloat16)
    s["v_cache"][slots // page, :, slots % page] = x[:, h_q + h_kv:].to(torch.bfloat16)
    return [q.to(torch.bfloat16), s["k_cache"], s["v_cache"]]


def _keys(s, cache, length):
    """[B, h_kv, length, D] in 32 bits, out of the pages."""
    case = s["case"]
    pages = _up(length, case["page"])
    got = cache[s["table"][:, :pages].clamp(min=0).long()]
    return got.permute(0, 2, 1, 3, 4).reshape(case["B"], case["h_kv"], -1, D)[:, :, :length].float()


def _visible(pos, key, window, n_sink):
    see = key <= pos
    return see & ((key > pos - window) | (key < n_sink)) if window else see


def _softmax_rows(x):
    """exp(x - max) and its sum along the last axis; a row of -inf alone gives zeros."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    e = (x - top).exp()
    return e, e.sum(-1, keepdim=True), top


def _plain_decode(s):
    case = s["case"]
    k, v = _keys(s, s["k_cache"], s["max_len"]), _keys(s, s["v_cache"], s["max_len"])
    q = s["q"].float().view(case["B"], case["h_kv"], -1, D)
    pos = s["seq_lens"].long()[:, None, None, None] - 1
    see = _visible(pos, torch.arange(s["max_len"], device=DEV), case["window"], case["n_sink"])
    x = (q @ k.transpose(-1, -2) * s["scale"]).masked_fill(~see, -torch.inf)
    e, total, _ = _softmax_rows(x)
    return (e @ v / total).to(torch.bfloat16).reshape(case["B"], case["h_q"], D)


def _plain_prompt(s):
    case, M = s["case"], s["max_new"]
    B, h_q, h_kv = case["B"], case["h_q"], case["h_kv"]
    cu = s["cu"].long()
    new = cu[1:] - cu[:-1]
    step = torch.arange(M, device=DEV)
    at = (cu[:-1, None] + step[None, :]).clamp(max=s["q"].shape[0] - 1)  # [B, M]: rows past a sequence are not kept
    q = s["q"][at].float().view(B, M, h_kv, -1, D).permute(0, 2, 3, 1, 4)  # [B, h_kv, G, M, D]
    k, v = _keys(s, s["k_cache"], s["max_len"])[:, :, None], _keys(s, s["v_cache"], s["max_len"])[:, :, None]
    pos = (s["seq_lens"].long() - new)[:, None] + step[None, :]
    see = _visible(pos[:, :, None], torch.arange(s["max_len"], device=DEV)[None, None, :], case["window"],
                   case["n_sink"])[:, None, None]
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~see, -torch.inf)
    top = x.amax(-1, keepdim=True)
    e = x.sub_(top).exp_()
    o = (e @ v / e.sum(-1, keepdim=True)).permute(0, 3, 1, 2, 4).reshape(B, M, h_q, D).to(torch.bfloat16)
    out = torch.empty_like(s["q"])
    seq = torch.searchsorted(cu[1:].contiguous(), torch.arange(out.shape[0], device=DEV), right=True)
    out[:] = o[seq, torch.arange(out.shape[0], device=DEV) - cu[seq]]
    return out


def _plain_prefix(s):
    case, n = s["case"], s["prefix"]
    B, h_kv, page = case["B"], case["h_kv"], case["page"]
    q = s["q"].float().view(B, h_kv, -1, D)
    # the prefix: every query against the same keys, as one product per key/value head
    flat = [c[s["prefix_table"].long()].permute(1, 0, 2, 3).reshape(h_kv, -1, D)[:, :n].float()
            for c in (s["k_cache"], s["v_cache"])]
    rows = q.transpose(0, 1).reshape(h_kv, -1, D)
    e1, l1, m1 = _softmax_rows(rows @ flat[0].transpose(-1, -2) * s["scale"])
    o1, l1, m1 = (t.reshape(h_kv, B, -1, t.shape[-1]).transpose(0, 1) for t in (e1 @ flat[1], l1, m1))
    # the sequences' own keys
    length = max(1, s["max_len"])
    k, v = _keys(s, s["k_cache"], length), _keys(s, s["v_cache"], length)
    see = torch.arange(length, device=DEV) < s["seq_lens"].long()[:, None, None, None]
    x = (q @ k.transpose(-1, -2) * s["scale"]).masked_fill(~see, -torch.inf)
    e2, l2, m2 = _softmax_rows(x)
    m2 = torch.where(l2 > 0, m2, -torch.inf)
    top = torch.maximum(m1, m2)
    a1, a2 = (m1 - top).exp(), (m2 - top).exp()
    o = (o1 * a1 + (e2 @ v) * a2) / (l1 * a1 + l2 * a2)
    return o.to(torch.bfloat16).reshape(B, case["h_q"], D)


# ---------------------------------------------------------------- the least work of a pass
def _seen(length, window, n_sink):
    """Keys the newest of `length` tokens sees."""
    if not window or length <= window:
        return length
    return window + min(n_sink, length - window)


def work(case):
    op = case["op"]
    if op == "plan":
        ctx, new = _lengths(case)
        fresh = sum(_up(c + n, case["page"]) - _up(c, case["page"]) for c, n in zip(ctx, new))
        cap = _up(sum(new), 64) * 64
        # the lengths; new pages read from the list and put into the table; a position and a slot per token row
        return dict(bytes=4 * (4 * case["B"] + 2 + 2 * fresh + 2 * cap), flops=8 * cap)
    if op == "qk":
        N, h_q, h_kv, rot = case["N"], case["h_q"], case["h_kv"], case["rot"]
        values = N * (h_q + 2 * h_kv) * D
        turned = N * (h_q + h_kv)
        return dict(bytes=2 * 2 * values + 8 * N + 2 * rot, flops=turned * (3 * rot + (4 * D if case["norm"] else 0)))
    ctx, new = _lengths(case)
    h_q, h_kv = case["h_q"], case["h_kv"]
    N = sum(new)
    window, n_sink = case.get("window", 0), case.get("n_sink", 0)
    pairs, rows = 0, 0
    for c, n in zip(ctx, new):
        if op == "prompt":
            if not window:
                pairs += n * c + n * (n + 1) // 2
                rows += c + n
            else:
                pairs += sum(_seen(p + 1, window, n_sink) for p in range(c, c + n))
                first = max(0, c + 1 - window)
                rows += c + n - first + min(n_sink, first)
        else:
            keys = _seen(c + 1, window, n_sink)
            pairs += keys
            rows += keys
    prefix = case.get("prefix", 0)
    return dict(bytes=2 * 2 * N * h_q * D + 2 * 2 * (rows + prefix) * h_kv * D,
                flops=4 * D * h_q * (pairs + N * prefix))


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "plan":
        return None
    if op == "qk":
        return _exact_qk(case, s)
    if work(case)["flops"] > 4e12:
        return None
    return _exact_attention(case, s)


def _exact_qk(case, s):
    h_q, h_kv, page, rot = case["h_q"], case["h_kv"], case["page"], case["rot"]
    N, half = case["N"], rot // 2
    x = s["qkv"].double().view(N, h_q + 2 * h_kv, D)
    parts = [x[:, :h_q].clone(), x[:, h_q:h_q + h_kv].clone()]
    theta = torch.outer(s["positions"].double(), s["inv_freq"].double())
    turn = torch.polar(torch.ones_like(theta), theta)[:, None, :]  # e^(i theta)
    for part, w in zip(parts, (s["q_weight"], s["k_weight"])):
        if w is not None:
            part.div_((part.square().sum(-1, keepdim=True) / D + s["eps"]).sqrt()).mul_(w.double())
        first = slice(0, rot, 2) if case["interleaved"] else slice(0, half)
        second = slice(1, rot, 2) if case["interleaved"] else slice(half, rot)
        z = torch.complex(part[..., first], part[..., second]) * turn
        part[..., first], part[..., second] = z.real.clone(), z.imag.clone()
    k, v = s["k_cache"].double(), s["v_cache"].double()
    rows = lambda c: c.transpose(1, 2).reshape(-1, h_kv, D)  # noqa: E731  (a copy, by slot)
    back = lambda r: r.view(-1, page, h_kv, D).transpose(1, 2).contiguous()  # noqa: E731
    rk, rv = rows(k), rows(v)
    rk[s["slots"].long()], rv[s["slots"].long()] = parts[1], x[:, h_q + h_kv:]
    return [parts[0], back(rk), back(rv)]


def _exact_attention(case, s):
    h_q, h_kv, page = case["h_q"], case["h_kv"], case["page"]
    group = h_q // h_kv
    ctx, new = _lengths(case)
    prefix, window, n_sink = case.get("prefix", 0), case.get("window", 0), case.get("n_sink", 0)
    table = s["table"].cpu().tolist()
    shared = s["prefix_table"].cpu().tolist() if prefix else []

    def fetch(cache, pages, j, n):
        return cache[pages, j].reshape(-1, D)[:n].double() if n else cache.new_zeros((0, D), dtype=torch.float64)

    out = torch.zeros(sum(new), h_q, D, dtype=torch.float64, device=DEV)
    head = [(fetch(s["k_cache"], shared, j, prefix), fetch(s["v_cache"], shared, j, prefix)) for j in range(h_kv)]
    row = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        length = c + n
        pages = table[b][:_up(length, page)]
        key = torch.arange(length, device=DEV)
        pos = torch.arange(c, c + n, device=DEV)[:, None]
        hidden = key > pos
        if window:
            hidden = hidden | ((key <= pos - window) & (key >= n_sink))
        for j in range(h_kv):
            k = torch.cat([head[j][0], fetch(s["k_cache"], pages, j, length)])
            v = torch.cat([head[j][1], fetch(s["v_cache"], pages, j, length)])
            for g in range(group) if n > 64 else [slice(0, group)]:
                at = j * group + g if n > 64 else slice(j * group, (j + 1) * group)
                q = s["q"][row:row + n, at].double()
                a = q @ k.T * s["scale"]
                cover = hidden if n > 64 else hidden[:, None, :]
                a[..., prefix:].masked_fill_(cover.expand(a[..., prefix:].shape), -torch.inf)
                out[row:row + n, at] = torch.softmax(a, -1) @ v
        row += n
    return out
