"""The operators of a serving step over a paged key/value cache, as measured workloads: maps of a
step (plan), rotary positions (rope), new rows into the cache (append), attention of the new tokens
over the pages (attn). `own` chooses between the library's calls and the plain torch forms."""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _plan(name, n, ctx, new, page, pad=0):
    return dict(name=name, op="plan", n=n, c_lo=ctx[0], c_hi=ctx[1], n_lo=new[0], n_hi=new[1],
                page=page, pad=pad)


def _rope(name, tokens, heads, d, rotary, pairs, ctx, packed, inverse=False, base=10000.0,
          factor=1.0, original=0):
    return dict(name=name, op="rope", tokens=tokens, heads=heads, d=d, rotary=rotary, pairs=pairs,
                ctx=ctx, packed=packed, inverse=inverse, base=base, factor=factor,
                original=original)


def _append(name, tokens, hq, hkv, d, rotary, pairs, page, ctx):
    return dict(name=name, op="append", tokens=tokens, hq=hq, hkv=hkv, d=d, rotary=rotary,
                pairs=pairs, page=page, ctx=ctx, base=10000.0, factor=1.0, original=0)


def _attn(name, n, q, k, hq, hkv, d, page, bias, causal=True, mixed=False, scale=None,
          buckets=32, distance=128):
    return dict(name=name, op="attn", n=n, q_lo=q[0], q_hi=q[1], k_lo=k[0], k_hi=k[1], hq=hq,
                hkv=hkv, d=d, page=page, bias=bias, causal=causal, mixed=mixed,
                scale=d ** -0.5 if scale is None else scale, buckets=buckets, distance=distance)


def listed():
    return [
        # the maps of one decode step: 64 requests, a token each, contexts of any length
        _plan("plan_decode_n64", 64, (1, 8192), (1, 1), 16),
        # the maps of a large mixed step: a thousand requests, from single tokens to prompts, and
        # a padded token count
        _plan("plan_mixed_n1000", 1000, (0, 16384), (1, 257), 64, pad=1000),
        # queries of a decode step, far positions, half of each head turned, halves layout
        _rope("rope_decode_t37_h32_d128", 37, 32, 128, 64, False, 131072, True),
        # queries of a long prompt, whole heads in pairs (the sizes of the rotary benchmark)
        _rope("rope_prompt_8x16384_h12_d64", 131072, 12, 64, 64, True, 16384, False),
        # gradient with frequencies stretched for a long context, from a packed projection
        _rope("rope_grad_t16383_h16_d128", 16383, 16, 128, 128, False, 65536, True, inverse=True,
              base=500000.0, factor=8.0, original=8192),
        # a decode step's new rows into the cache, queries turned on the way
        _append("append_t48_h32x8_d128", 48, 32, 8, 128, 128, False, 16, 32768),
        # a prompt chunk's rows
        _append("append_t8192_h16x4_d128", 8192, 16, 4, 128, 128, True, 64, 16384),
        # the smallest call: one token of one request, a short context, the T5 decoder's bias
        _attn("attn_one_b1_k500_h12_d64", 1, (1, 1), (500, 500), 12, 12, 64, 16, "t5", scale=1.0),
        # decode over ragged contexts, grouped heads, linear bias
        _attn("attn_decode_b32_k4096_h64x16_d128", 32, (1, 1), (1024, 4096), 64, 16, 128, 64,
              "alibi"),
        # a few drafted tokens for each request, odd group, T5 bias
        _attn("attn_draft_b24_q5_k6000_h24x8_d64", 24, (5, 5), (600, 6000), 24, 8, 64, 32, "t5"),
        # a step that mixes single tokens with one prompt chunk
        _attn("attn_mixed_b25_q384_k6000_h16x4_d128", 25, (1, 384), (300, 6000), 16, 4, 128, 16,
              "none", mixed=True),
        # a prompt chunk over a long context, linear bias
        _attn("attn_chunk_q2048_k18432_h16x8_d128", 1, (2048, 2048), (18432, 18432), 16, 8, 128,
              128, "alibi"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _cost(c):
    """Values that the plain form holds at once: what a drawn case is bounded by."""
    if c["op"] == "plan":
        return c["n"] * (_pages(c) + c["n_hi"])
    if c["op"] == "rope":
        return c["tokens"] * c["heads"] * c["d"]
    if c["op"] == "append":
        return c["tokens"] * (c["hq"] + 2 * c["hkv"]) * c["d"]
    return (c["n"] * c["q_hi"] * c["k_hi"] * c["hq"]
            + 4 * c["n"] * c["k_hi"] * (c["hkv"] * c["d"]) + c["n"] * c["q_hi"] * c["hq"] * c["d"])


def draw(rng):
    op = rng.choice(["plan", "rope", "append", "attn", "attn", "attn"])
    limit = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        d = rng.choice([64, 128])
        page = rng.choice([16, 32, 64, 128, 256])
        pairs = rng.random() < 0.5
        rotary = rng.choice([d // 4, d // 2, d, d])
        if op == "plan":
            n_lo = _log_int(rng, 1, 16)
            c = _plan("", _log_int(rng, 1, 1024), (rng.choice([0, 1, 100]), _log_int(rng, 128, 32768)),
                      (n_lo, max(n_lo, _log_int(rng, 1, 256))), page, rng.choice([0, 17, 256]))
        elif op == "rope":
            c = _rope("", _log_int(rng, 1, 65536), _log_int(rng, 1, 64), d, rotary, pairs,
                      _log_int(rng, 1024, 262144), rng.random() < 0.5, rng.random() < 0.5,
                      rng.choice([500.0, 10000.0, 500000.0]), rng.choice([1.0, 4.0]),
                      rng.choice([0, 4096]))
        elif op == "append":
            hkv = _log_int(rng, 1, 16)
            c = _append("", _log_int(rng, 1, 16384), hkv * rng.choice([1, 2, 3, 4, 8]), hkv, d,
                        rotary, pairs, page, _log_int(rng, 1024, 65536))
        else:
            hkv = _log_int(rng, 1, 16)
            q_lo = rng.choice([1, 1, 1, _log_int(rng, 2, 16), _log_int(rng, 8, 1024)])
            q_hi = q_lo if rng.random() < 0.5 else _log_int(rng, q_lo, 4 * q_lo + 8)
            k_lo = _log_int(rng, q_hi, q_hi + 1000)
            c = _attn("", _log_int(rng, 1, 64), (q_lo, q_hi), (k_lo, _log_int(rng, k_lo, k_lo + 32768)),
                      hkv * rng.choice([1, 2, 3, 4, 5, 8, 16]), hkv, d, page,
                      rng.choice(["none", "t5", "alibi", "both"]), causal=rng.random() < 0.8,
                      mixed=rng.random() < 0.3, buckets=rng.choice([32, 64]),
                      distance=rng.choice([128, 1024]))
        if _cost(c) <= limit:
            del c["name"]
            return c


def _lengths(lo, hi, n, phase):
    """n lengths spread evenly over the logarithm of lo..hi, in an order that looks random."""
    lo = max(lo, 0)
    x = (phase + 0.6180339887498949 * np.arange(1, n + 1)) % 1.0
    v = np.exp(np.log(lo + 1) + x * (np.log(hi + 1) - np.log(lo + 1))) - 1
    v = np.clip(np.rint(v), lo, hi).astype(np.int64)
    v[0] = hi  # the bound is reached
    return v


def _attn_lengths(c):
    if c["mixed"]:
        new = np.full(c["n"], c["q_lo"], np.int64)
        new[0] = c["q_hi"]
    else:
        new = _lengths(c["q_lo"], c["q_hi"], c["n"], 0.25)
    return new, np.maximum(_lengths(c["k_lo"], c["k_hi"], c["n"], 0.0), new)


def _plan_lengths(c):
    return _lengths(c["c_lo"], c["c_hi"], c["n"], 0.5), _lengths(c["n_lo"], c["n_hi"], c["n"], 0.125)


def _pages(c):
    return -(-(c["c_hi"] + c["n_hi"]) // c["page"])


def work(case):
    c = case
    if c["op"] == "plan":
        ctx, new = _plan_lengths(c)
        pages = int((-(-(ctx + new) // c["page"]) - -(-ctx // c["page"])).sum())
        tokens = int(new.sum()) + c["pad"]
        ints = 2 * c["n"] + 2 * pages + 2 * c["n"] + 3 + 2 * tokens
        return {"bytes": 4 * ints, "flops": 0}
    if c["op"] == "rope":
        values = c["tokens"] * c["heads"] * c["d"]
        return {"bytes": 4 * values + 4 * c["tokens"],
                "flops": 3 * c["tokens"] * c["heads"] * c["rotary"]}
    if c["op"] == "append":
        values = c["tokens"] * (c["hq"] + 2 * c["hkv"]) * c["d"]
        return {"bytes": 4 * values + 8 * c["tokens"],
                "flops": 3 * c["tokens"] * (c["hq"] + c["hkv"]) * c["rotary"]}
    new, ctx = _attn_lengths(c)
    if c["causal"]:  # query j of a request sees its keys 0 .. lk - lq + j
        seen = int((new * (ctx - new) + new * (new + 1) // 2).sum())
    else:
        seen = int((new * ctx).sum())
    tq = int(new.sum())
    return {"bytes": int(ctx.sum()) * c["hkv"] * c["d"] * 4 + tq * c["hq"] * (4 * c["d"] + 4),
            "flops": 4 * seen * c["hq"] * c["d"]}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _ints(v, dev="cuda"):
    return torch.as_tensor(np.ascontiguousarray(v, dtype=np.int32), device=dev)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _turns(c):
    """Turned frequencies of each pair (64 bits): base^(-2i/r), between the wavelengths that fit
    the original length four times and once blended into their factor-th part; without an
    original length all of them divided by the factor."""
    i = torch.arange(c["rotary"] // 2, dtype=torch.float64, device="cuda")
    theta = torch.exp(-2.0 * i / c["rotary"] * math.log(c["base"]))
    if c["original"] == 0:
        return theta / c["factor"]
    keep = ((c["original"] * theta / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
    return theta * (keep + (1.0 - keep) / c["factor"])


def _edges(c):
    """Distances at which the T5 bucket of one direction moves on, by whole numbers: the first n
    with n^E e^t >= D^t e^E (e exact buckets, E logarithmic ones, D the maximum distance)."""
    per = c["buckets"]  # a decoder's buckets: one direction
    e = per // 2
    top = per - e
    first = [next(n for n in range(e, c["distance"] + 1)
                  if n ** top * e ** t >= c["distance"] ** t * e ** top) for t in range(1, top)]
    return torch.tensor(list(range(1, e + 1)) + first, device="cuda", dtype=torch.int64)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "plan":
        ctx, new = _plan_lengths(c)
        have = -(-ctx // c["page"])
        need = -(-(ctx + new) // c["page"]) - have
        width = _pages(c)
        pool = int((have + need).sum()) + 64
        order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        first = torch.as_tensor(np.cumsum(have) - have, device="cuda")
        col = torch.arange(width, device="cuda")
        hv = torch.as_tensor(have, device="cuda")[:, None]
        at = (first[:, None] + col[None]).clamp(max=pool - 1)
        s["table"] = torch.where(col[None] < hv, order[at], -1).to(torch.int32).contiguous()
        s.update(ctx=_ints(ctx), new=_ints(new), free=order[int(have.sum()):].contiguous(),
                 pool=pool, tokens=int(new.sum()) + c["pad"])
        n, t = c["n"], s["tokens"]
        for k, m in (("cu", n + 1), ("lk", n), ("pos", t), ("slots", t), ("counts", 2)):
            s[k] = torch.zeros(m, dtype=torch.int32, device="cuda")
        return s
    if c["op"] in ("rope", "append"):
        t = c["tokens"]
        s["pos"] = torch.randint(0, c["ctx"], (t,), generator=g, device="cuda").to(torch.int32)
        s["theta"] = _turns(c)
        if own:
            import attention_relative_position_gb300 as fa
            s["rope"] = fa.fat_rope_init(c["rotary"], base=c["base"], interleaved=c["pairs"],
                                         factor=c["factor"],
                                         ramp=(1.0, 4.0, c["original"]) if c["original"] else None)
        if c["op"] == "rope":  # the queries of a packed projection, or rows of their own
            wide = c["heads"] + (2 * max(1, c["heads"] // 4) if c["packed"] else 0)
            s["x"] = _normal(g, t, wide, c["d"])[:, :c["heads"]]
            s["out"] = torch.empty(t, c["heads"], c["d"], dtype=torch.bfloat16, device="cuda")
            return s
        qkv = _normal(g, t, c["hq"] + 2 * c["hkv"], c["d"])
        s["q"], s["k"], s["v"] = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=1)
        pages = 2 * -(-t // c["page"]) + 1
        s["kc"] = _normal(g, pages, c["page"], c["hkv"], c["d"])
        s["vc"] = _normal(g, pages, c["page"], c["hkv"], c["d"])
        s["slots"] = torch.randperm(pages * c["page"], generator=g, device="cuda")[:t].to(torch.int32)
        s["q_out"] = torch.empty(t, c["hq"], c["d"], dtype=torch.bfloat16, device="cuda")
        return s
    new, ctx = _attn_lengths(c)
    used = -(-ctx // c["page"])
    width = int(used.max())
    pool = int(used.sum()) + 3
    order = torch.randperm(pool, generator=g, device="cuda")
    first = torch.as_tensor(np.cumsum(used) - used, device="cuda")
    col = torch.arange(width, device="cuda")
    held = col[None] < torch.as_tensor(used, device="cuda")[:, None]
    s["table"] = torch.where(held, order[(first[:, None] + col[None]).clamp(max=pool - 1)], 0)
    s["table"] = s["table"].to(torch.int32).contiguous()
    s["kc"] = _normal(g, pool, c["page"], c["hkv"], c["d"])
    s["vc"] = _normal(g, pool, c["page"], c["hkv"], c["d"])
    s["q"] = _normal(g, int(new.sum()), c["hq"], c["d"])
    if c["scale"] == 1.0:  # T5 takes no scale: its queries are that much smaller
        s["q"] = (s["q"].float() * c["d"] ** -0.5).to(torch.bfloat16)
    s["cu"] = _ints(np.concatenate([[0], np.cumsum(new)]))
    s["lk"] = _ints(ctx)
    s["max_q"], s["max_k"] = int(new.max()), int(ctx.max())
    s["bias"], s["slopes"] = None, None
    if c["bias"] in ("t5", "both"):
        s["bias"] = 0.5 * torch.randn(c["buckets"], c["hq"], generator=g, device="cuda")
        s["edges"] = _edges(c)
    if c["bias"] in ("alibi", "both"):
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["hq"] + 1, device="cuda") / c["hq"]).float()
    if own:
        import attention_relative_position_gb300 as fa
        size = fa.fat_paged_attn_workspace_size(s["q"], s["kc"], s["cu"], s["max_q"], s["max_k"])
        s["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import attention_relative_position_gb300 as fa
    c = s["case"]
    if c["op"] == "plan":
        cu, lk, pos, slots, counts = fa.fat_paged_plan(
            s["ctx"], s["new"], s["free"], s["table"], c["page"], s["pool"], s["tokens"],
            cu_seqlens_q=s["cu"], seqlens_k=s["lk"], positions=s["pos"], slots=s["slots"],
            counts=s["counts"])
        return {"table": s["table"], "cu": cu, "lk": lk, "pos": pos, "slots": slots,
                "counts": counts}
    if c["op"] == "rope":
        return fa.fat_rope_embed(s["x"], s["pos"], s["rope"], inverse=c["inverse"], out=s["out"])
    if c["op"] == "append":
        fa.fat_paged_append(s["k"], s["v"], s["kc"], s["vc"], s["slots"], q=s["q"],
                            positions=s["pos"], rope=s["rope"], q_out=s["q_out"])
        return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}
    out, lse = fa.fat_paged_attn(
        s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["lk"], s["max_q"], s["max_k"],
        bias_table=s["bias"], num_buckets=c["buckets"], max_distance=c["distance"],
        bidirectional=False, alibi_slopes=s["slopes"], causal=c["causal"],
        softmax_scale=c["scale"], workspace=s["ws"])
    return {"out": out, "lse": lse}


def _rotated(x, pos, theta, pairs, inverse=False):
    """Rows of x (fp32) turned by pos * theta; angles in 64 bits."""
    r = 2 * theta.numel()
    angle = pos.double()[:, None] * theta[None]
    cs, sn = angle.cos().float()[:, None], angle.sin().float()[:, None]
    sn = -sn if inverse else sn
    head, rest = x[..., :r], x[..., r:]
    if pairs:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * cs - b * sn, a * sn + b * cs], dim=-1).flatten(-2)
    else:
        a, b = head[..., :r // 2], head[..., r // 2:]
        turned = torch.cat([a * cs - b * sn, a * sn + b * cs], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "plan":
        return _plan_plain(s, c)
    if c["op"] == "rope":
        y = _rotated(s["x"].float(), s["pos"], s["theta"], c["pairs"], c["inverse"])
        return y.to(torch.bfloat16)
    if c["op"] == "append":
        at = s["slots"].long()
        q = _rotated(s["q"].float(), s["pos"], s["theta"], c["pairs"]).to(torch.bfloat16)
        k = _rotated(s["k"].float(), s["pos"], s["theta"], c["pairs"]).to(torch.bfloat16)
        s["kc"].view(-1, c["hkv"], c["d"])[at] = k
        s["vc"].view(-1, c["hkv"], c["d"])[at] = s["v"]
        return {"q": q, "k": s["kc"], "v": s["vc"]}
    return _attn_plain(s, c)


def _plan_plain(s, c):
    page, n = c["page"], c["n"]
    ctx, new = s["ctx"].long(), s["new"].long()
    lk = ctx + new
    have = (ctx + page - 1) // page
    need = (lk + page - 1) // page - have
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    cu = torch.cat([zero, new.cumsum(0)])
    first = need.cumsum(0) - need
    j = torch.arange(s["table"].shape[1], device="cuda")[None] - have[:, None]
    fresh = s["free"][(first[:, None] + j).clamp(0, s["free"].numel() - 1)]
    table = torch.where((j >= 0) & (j < need[:, None]), fresh, s["table"])
    t = torch.arange(s["tokens"], device="cuda")
    i = torch.searchsorted(cu, t, right=True) - 1
    real = i < n
    i = i.clamp(max=n - 1)
    pos = ctx[i] + t - cu[i]
    column = (pos // page).clamp(max=table.shape[1] - 1)
    slot = torch.where(real, table[i, column].long() * page + pos % page, -1)
    pos = torch.where(real, pos, 0)
    counts = torch.stack([need.sum(), new.sum()])
    return {"table": table, "cu": cu.int(), "lk": lk.int(), "pos": pos.int(), "slots": slot.int(),
            "counts": counts.int()}


def _attn_plain(s, c):
    n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
    group, mq, mk = hq // hkv, s["max_q"], s["max_k"]
    cu, lk = s["cu"].long(), s["lk"].long()
    lq = cu[1:] - cu[:-1]
    j = torch.arange(mq, device="cuda")
    row = (cu[:-1, None] + j[None]).clamp(max=s["q"].shape[0] - 1)
    kpos = torch.arange(mk, device="cuda")
    table = s["table"].long()
    k = s["kc"][table].flatten(1, 2)[:, :mk].float().permute(0, 2, 3, 1)
    v = s["vc"][table].flatten(1, 2)[:, :mk].float().transpose(1, 2)
    q = s["q"][row].float().view(n, mq, hkv, group, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(n, hkv, group * mq, d), k).view(n, hkv, group, mq, mk)
    x = x.mul_(c["scale"])
    qpos = (lk - lq)[:, None] + j[None]
    delta = kpos[None, None] - qpos[:, :, None]  # [n, mq, mk]
    if s["bias"] is not None:
        bucket = torch.bucketize((-delta).clamp(min=0), s["edges"], right=True)
        x += s["bias"].t()[:, bucket].view(hkv, group, n, mq, mk).permute(2, 0, 1, 3, 4)
    if s["slopes"] is not None:
        far = delta.abs().float().view(n, 1, 1, mq, mk)
        x -= s["slopes"].view(1, hkv, group, 1, 1) * far
    hide = kpos[None, None] >= lk[:, None, None]
    if c["causal"]:
        hide = hide | (delta > 0)
    x.masked_fill_(hide.view(n, 1, 1, mq, mk), float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, hkv, group * mq, mk), v).view(n, hkv, group, mq, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (total.log() + top).squeeze(-1)
    t = torch.arange(s["q"].shape[0], device="cuda")
    i = torch.searchsorted(cu, t, right=True) - 1
    o = o.permute(0, 3, 1, 2, 4).reshape(n, mq, hq, d)[i, t - cu[i]]
    lse = lse.permute(0, 3, 1, 2).reshape(n, mq, hq)[i, t - cu[i]]
    return {"out": o.to(torch.bfloat16), "lse": lse.t().contiguous()}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, request by request
# ---------------------------------------------------------------------------------------------
def _bucket_exact(n, per, far):
    """T5 bucket of distance n >= 0: n itself below per // 2, then the largest t < E with
    (n / e)^E >= (far / e)^t, both sides whole numbers."""
    e = per // 2
    top = per - e
    if n < e:
        return n
    t = 0
    while t + 1 < top and n ** top * e ** (t + 1) >= far ** (t + 1) * e ** top:
        t += 1
    return e + t


def _turn_exact(x, pos, c, inverse):
    r = c["rotary"]
    y = x.clone()
    sign = -1.0 if inverse else 1.0
    for i in range(r // 2):
        theta = c["base"] ** (-2.0 * i / r)
        if c["original"]:
            turns = c["original"] * theta / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / 3.0))
            theta = theta * keep + theta * (1.0 - keep) / c["factor"]
        else:
            theta = theta / c["factor"]
        angle = pos.double() * theta
        cs, sn = torch.cos(angle)[:, None], sign * torch.sin(angle)[:, None]
        a, b = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + r // 2)
        y[..., a] = x[..., a] * cs - x[..., b] * sn
        y[..., b] = x[..., a] * sn + x[..., b] * cs
    return y


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "plan":
        return _plan_exact(s, c)
    if c["op"] == "rope":
        return _turn_exact(s["x"].double(), s["pos"], c, c["inverse"])
    if c["op"] == "append":
        k, v = s["kc"].double(), s["vc"].double()
        page, at = c["page"], s["slots"].long()
        k[at // page, at % page] = _turn_exact(s["k"].double(), s["pos"], c, False)
        v[at // page, at % page] = s["v"].double()
        return {"q": _turn_exact(s["q"].double(), s["pos"], c, False), "k": k, "v": v}
    new, ctx = _attn_lengths(c)
    hq, group = c["hq"], c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((hq, s["q"].shape[0]), float("-inf"), dtype=torch.float64, device="cuda")
    by_distance = None
    if s["bias"] is not None:
        ids = [_bucket_exact(n, c["buckets"], c["distance"]) for n in range(c["distance"] + 1)]
        by_distance = s["bias"].double()[torch.tensor(ids, device="cuda")]  # [distance, hq]
    at = 0
    for i in range(c["n"]):
        lq, lk = int(new[i]), int(ctx[i])
        pages = s["table"][i, :-(-lk // c["page"])].long()
        keys = s["kc"][pages].flatten(0, 1)[:lk].double()
        values = s["vc"][pages].flatten(0, 1)[:lk].double()
        dist = (lk - lq + torch.arange(lq, device="cuda"))[:, None] - torch.arange(lk, device="cuda")
        for h in range(hq):
            x = c["scale"] * (s["q"][at:at + lq, h].double() @ keys[:, h // group].t())
            if by_distance is not None:
                x = x + by_distance[:, h][dist.clamp(0, c["distance"])]
            if s["slopes"] is not None:
                x = x - float(s["slopes"][h]) * dist.abs().double()
            if c["causal"]:
                x = x.masked_fill(dist < 0, float("-inf"))
            lse[h, at:at + lq] = torch.logsumexp(x, dim=-1)
            out[at:at + lq, h] = torch.softmax(x, dim=-1) @ values[:, h // group]
        at += lq
    return {"out": out, "lse": lse}


def _plan_exact(s, c):
    ctx, new = _plan_lengths(c)
    page = c["page"]
    table, free = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy()
    cu, pos, slots, taken = [0], [], [], 0
    for i in range(c["n"]):
        total = int(ctx[i] + new[i])
        for column in range(-(-int(ctx[i]) // page), -(-total // page)):
            table[i, column] = free[taken]
            taken += 1
        for p in range(int(ctx[i]), total):
            pos.append(p)
            slots.append(int(table[i, p // page]) * page + p % page)
        cu.append(len(pos))
    pos += [0] * c["pad"]
    slots += [-1] * c["pad"]
    as_int = lambda v: np.asarray(v, dtype=np.int32)  # noqa: E731
    return {"table": table, "cu": as_int(cu), "lk": as_int(ctx + new), "pos": as_int(pos),
            "slots": as_int(slots), "counts": as_int([taken, cu[-1]])}
