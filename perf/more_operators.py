"""The output layer's loss without its logits and attention over trees of drafted tokens, as measured
workloads: the loss of hidden rows over a vocabulary (loss; with few rows the scores of drafted
tokens), its gradient (grad), the maps of trees of drafted tokens (tree_plan) and their attention over
a paged key/value cache (tree_attn). `own` chooses between the library's calls and the plain torch
forms."""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _head(op, name, rows, vocab, dim, z=0.0, tied=False, ignored=0.0, weighted=False):
    return dict(name=name, op=op, rows=rows, vocab=vocab, dim=dim, z=z, tied=tied, ignored=ignored,
                weighted=weighted)


def _tree_plan(name, n, q, ctx, reach, pad=0):
    return dict(name=name, op="tree_plan", n=n, q_lo=q[0], q_hi=q[1], c_lo=ctx[0], c_hi=ctx[1],
                reach=reach, pad=pad)


def _tree_attn(name, n, q, ctx, hq, hkv, d, page, bias, reach, buckets=32, distance=128):
    return dict(name=name, op="tree_attn", n=n, q_lo=q[0], q_hi=q[1], c_lo=ctx[0], c_hi=ctx[1],
                hq=hq, hkv=hkv, d=d, page=page, bias=bias, reach=reach,
                scale=1.0 if bias == "t5" else d ** -0.5, buckets=buckets, distance=distance)


def listed():
    return [
        # the smallest call: the score of one drafted token, the layer's weights read once
        _head("loss", "score_t1_v32768_d512", 1, 32768, 512),
        # an odd batch over an odd vocabulary, tied embeddings (scaled logits), padding ignored
        _head("loss", "loss_t2077_v50021_d776", 2077, 50021, 776, z=1e-4, tied=True, ignored=0.2),
        # the loss of a training or validation batch (rows and vocabulary of the loss benchmark)
        _head("loss", "loss_t8192_v32768_d1024", 8192, 32768, 1024, z=1e-4),
        # gradient of a small odd batch, a weight for each token
        _head("grad", "grad_t517_v32003_d776", 517, 32003, 776, z=1e-4, tied=True, ignored=0.2,
              weighted=True),
        # gradient of the training batch above
        _head("grad", "grad_t8192_v32768_d1024", 8192, 32768, 1024, z=1e-4),
        # gradient over a large vocabulary: logits of 1 GB that are not kept
        _head("grad", "grad_t4096_v131072_d2048", 4096, 131072, 2048, ignored=0.05),
        # the maps of a step that verifies the trees of 16 requests
        _tree_plan("tree_plan_n16_q64", 16, (64, 64), (100, 8192), 8),
        # of many requests with trees of all sizes, long paths, a padded token count
        _tree_plan("tree_plan_n512_q256", 512, (1, 256), (0, 16384), 2, pad=777),
        # the smallest call: one request's tree over a short context, the T5 decoder's bias
        _tree_attn("tree_attn_b1_q26_k700_h12_d64", 1, (26, 26), (700, 700), 12, 12, 64, 16, "t5", 8),
        # few tokens a request, head groups of three
        _tree_attn("tree_attn_b24_q5_k6000_h24x8_d64", 24, (5, 5), (600, 6000), 24, 8, 64, 32,
                   "none", 3),
        # trees of 12 tokens, ragged contexts, linear bias
        _tree_attn("tree_attn_b64_q12_k4096_h16x4_d128", 64, (12, 12), (1024, 4096), 16, 4, 128, 64,
                   "alibi", 4),
        # large trees of all sizes over long contexts
        _tree_attn("tree_attn_b16_q61_k6000_h32x8_d128", 16, (24, 61), (1500, 6000), 32, 8, 128, 64,
                   "none", 8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _cost(c):
    if c["op"] in ("loss", "grad"):
        return c["rows"] * c["vocab"] * c["dim"]
    if c["op"] == "tree_plan":
        return c["n"] * c["q_hi"] * c["q_hi"]
    keys = c["n"] * (c["c_hi"] + c["q_hi"])
    return keys * c["q_hi"] * c["hq"] + 4 * keys * c["hkv"] * c["d"]


def draw(rng):
    op = rng.choice(["loss", "grad", "loss", "grad", "tree_plan", "tree_attn", "tree_attn"])
    limit = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        if op in ("loss", "grad"):
            c = _head(op, "", _log_int(rng, 1, 16384), _log_int(rng, 300, 131072),
                      8 * _log_int(rng, 8, 512), z=rng.choice([0.0, 1e-4]),
                      tied=rng.random() < 0.3, ignored=rng.choice([0.0, 0.0, 0.3]),
                      weighted=op == "grad" and rng.random() < 0.4)
        else:
            lo = _log_int(rng, 1, 64)
            q = (lo, lo if rng.random() < 0.5 else _log_int(rng, lo, 4 * lo))
            c_lo = _log_int(rng, 1, 2000)
            ctx = (c_lo, _log_int(rng, c_lo + 100, c_lo + 16384))
            n = _log_int(rng, 1, 512 if op == "tree_plan" else 64)
            reach = rng.choice([1, 2, 4, 16])
            if op == "tree_plan":
                c = _tree_plan("", n, q, ctx, reach, rng.choice([0, 5, 300]))
            else:
                hkv = _log_int(rng, 1, 16)
                c = _tree_attn("", n, q, ctx, hkv * rng.choice([1, 2, 3, 4, 8]), hkv,
                               rng.choice([64, 128]), rng.choice([16, 32, 64, 128]),
                               rng.choice(["none", "t5", "alibi"]), reach,
                               buckets=rng.choice([32, 64]), distance=rng.choice([128, 1024]))
        if _cost(c) <= limit:
            del c["name"]
            return c


def _lengths(lo, hi, n, phase):
    """n lengths spread evenly over the logarithm of lo..hi, in an order that looks random."""
    x = (phase + 0.6180339887498949 * np.arange(1, n + 1)) % 1.0
    v = np.exp(np.log(lo + 1) + x * (np.log(hi + 1) - np.log(lo + 1))) - 1
    v = np.clip(np.rint(v), lo, hi).astype(np.int64)
    v[0] = hi  # the bound is reached
    return v


def _tree_lengths(c):
    """Nodes and cached tokens of every request."""
    return _lengths(c["q_lo"], c["q_hi"], c["n"], 0.25), _lengths(c["c_lo"], c["c_hi"], c["n"], 0.0)


def work(case):
    c = case
    if c["op"] == "loss":
        values = (c["rows"] + c["vocab"]) * c["dim"]
        return {"bytes": 2 * values + 12 * c["rows"],
                "flops": 2 * c["rows"] * c["vocab"] * c["dim"]}
    if c["op"] == "grad":
        values = (c["rows"] + c["vocab"]) * c["dim"]
        return {"bytes": 4 * values + (12 if c["weighted"] else 8) * c["rows"],
                "flops": 6 * c["rows"] * c["vocab"] * c["dim"]}
    new, ctx = _tree_lengths(c)
    tq = int(new.sum())
    if c["op"] == "tree_plan":
        words = -(-c["q_hi"] // 32)
        return {"bytes": 4 * (tq + 2 * c["n"] + 1 + (tq + c["pad"]) * (1 + words)), "flops": 0}
    # every node sees its request's context, and about its depth of the other nodes
    return {"bytes": int((ctx + new).sum()) * c["hkv"] * c["d"] * 4 + tq * c["hq"] * (4 * c["d"] + 4),
            "flops": 4 * int((new * ctx).sum()) * c["hq"] * c["d"]}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _ints(v, dev="cuda"):
    return torch.as_tensor(np.ascontiguousarray(v, dtype=np.int32), device=dev)


def _normal(g, *shape, std=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (x * std).to(torch.bfloat16)


def _trees(new, reach, seed):
    """Parents of every request's nodes: node 0 follows the context, node j one of the `reach` nodes
    before it (1: a chain)."""
    r = np.random.default_rng(seed)
    out = []
    for m in new:
        j = np.arange(int(m))
        out.append(np.where(j == 0, -1, j - 1 - np.minimum(r.integers(0, reach, int(m)), j - 1)))
    return np.concatenate(out)


def _contexts(c, ctx, seed):
    """Cached tokens: for the maps, whose work does not depend on them, drawn anew."""
    if c["op"] != "tree_plan":
        return ctx
    return np.random.default_rng([int(seed), 1]).integers(c["c_lo"], c["c_hi"] + 1, len(ctx))


def _paths(parents, new):
    """Depth of every node, and its path as (node, ancestor) pairs, itself among them."""
    depth, pairs, at = np.zeros(len(parents), np.int64), [], 0
    for m in new:
        path = []
        for j in range(int(m)):
            p = int(parents[at + j])
            path.append((path[p] if p >= 0 else []) + [j])
            depth[at + j] = len(path[j]) - 1
            pairs.append(path[j])
        at += int(m)
    return depth, pairs


def _words(pairs, words):
    out = np.zeros((len(pairs), words), np.uint32)
    for i, path in enumerate(pairs):
        for j in path:
            out[i, j >> 5] |= np.uint32(1 << (j & 31))
    return out.view(np.int32)


def _edges(c):
    """Distances at which the T5 bucket of one direction moves on, by whole numbers: the first n
    with n^E e^t >= D^t e^E (e exact buckets, E logarithmic ones, D the maximum distance)."""
    e = c["buckets"] // 2  # a decoder's buckets: one direction
    top = c["buckets"] - e
    first = [next(n for n in range(e, c["distance"] + 1)
                  if n ** top * e ** t >= c["distance"] ** t * e ** top) for t in range(1, top)]
    return torch.tensor(list(range(1, e + 1)) + first, device="cuda", dtype=torch.int64)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    if c["op"] in ("loss", "grad"):
        n, v, d = c["rows"], c["vocab"], c["dim"]
        # normalised rows, and logits of a standard deviation of about 2; tied embeddings are as
        # large as the rows, and the logits scaled instead
        s["hidden"] = _normal(g, n, d)
        s["weight"] = _normal(g, v, d, std=2.0 if c["tied"] else 2.0 * d ** -0.5)
        s["scale"] = d ** -0.5 if c["tied"] else 1.0
        s["target"] = torch.randint(0, v, (n,), generator=g, device="cuda").to(torch.int32)
        drop = torch.rand(n, generator=g, device="cuda") < c["ignored"]
        s["target"] = torch.where(drop, -100, s["target"]).to(torch.int32)
        s["dloss"] = torch.rand(n, generator=g, device="cuda") if c["weighted"] else None
        s["grad_scale"] = 1.0 / n
        if c["op"] == "grad":  # the forward's statistics
            s["lse"] = torch.cat([torch.logsumexp(z, -1) for _, z in _logit_rows(s)])
            s["dweight"] = torch.empty(v, d, dtype=torch.bfloat16, device="cuda")
        if own:
            import attention_relative_position_gb300 as fa
            size = fa.fat_linear_cross_entropy_workspace_size(n, v, d, backward=c["op"] == "grad")
            s["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
        return s
    new, ctx = _tree_lengths(c)
    ctx = _contexts(c, ctx, seed)
    parents = _trees(new, c["reach"], int(seed))
    tq = int(new.sum())
    s["cu"], s["lk"] = _ints(np.concatenate([[0], np.cumsum(new)])), _ints(ctx + new)
    s["max_q"], s["max_k"] = int(new.max()), int((ctx + new).max())
    words = -(-c["q_hi"] // 32)
    if c["op"] == "tree_plan":
        t = tq + c["pad"]
        s["parents"] = _ints(np.concatenate([parents, np.zeros(c["pad"], np.int64)]))
        s["positions"] = torch.zeros(t, dtype=torch.int32, device="cuda")
        s["mask"] = torch.zeros(t, words, dtype=torch.int32, device="cuda")
        return s
    depth, pairs = _paths(parents, new)
    s["positions"] = _ints(np.repeat(ctx, new) + depth)
    s["mask"] = torch.as_tensor(_words(pairs, words), device="cuda")
    used = -(-(ctx + new) // c["page"])
    pool = int(used.sum()) + 3
    order = torch.randperm(pool, generator=g, device="cuda")
    first = torch.as_tensor(np.cumsum(used) - used, device="cuda")
    col = torch.arange(int(used.max()), device="cuda")
    held = col[None] < torch.as_tensor(used, device="cuda")[:, None]
    s["table"] = torch.where(held, order[(first[:, None] + col[None]).clamp(max=pool - 1)], 0)
    s["table"] = s["table"].to(torch.int32).contiguous()
    s["kc"] = _normal(g, pool, c["page"], c["hkv"], c["d"])
    s["vc"] = _normal(g, pool, c["page"], c["hkv"], c["d"])
    # T5 takes no scale: its queries are that much smaller
    s["q"] = _normal(g, tq, c["hq"], c["d"], std=c["d"] ** -0.5 if c["scale"] == 1.0 else 1.0)
    s["bias"], s["slopes"] = None, None
    if c["bias"] == "t5":
        s["bias"] = 0.5 * torch.randn(c["buckets"], c["hq"], generator=g, device="cuda")
        s["edges"] = _edges(c)
    if c["bias"] == "alibi":
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
    if c["op"] == "loss":
        loss, lse = fa.fat_linear_cross_entropy_fwd(
            s["hidden"], s["weight"], s["target"], z_loss=c["z"], logit_scale=s["scale"],
            workspace=s["ws"])
        return {"loss": loss, "lse": lse}
    if c["op"] == "grad":
        dhidden, dweight = fa.fat_linear_cross_entropy_bwd(
            s["hidden"], s["weight"], s["target"], s["lse"], dloss=s["dloss"], z_loss=c["z"],
            logit_scale=s["scale"], grad_scale=s["grad_scale"], dweight=s["dweight"],
            workspace=s["ws"])
        return {"dhidden": dhidden, "dweight": dweight}
    if c["op"] == "tree_plan":
        positions, mask = fa.fat_paged_tree_plan(s["parents"], s["cu"], s["lk"], c["q_hi"],
                                                 positions=s["positions"], tree_mask=s["mask"])
        return {"positions": positions, "mask": mask}
    out, lse = fa.fat_paged_tree_attn(
        s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["lk"], s["positions"], s["mask"],
        s["max_q"], s["max_k"], bias_table=s["bias"], num_buckets=c["buckets"],
        max_distance=c["distance"], bidirectional=False, alibi_slopes=s["slopes"],
        softmax_scale=c["scale"], workspace=s["ws"])
    return {"out": out, "lse": lse}


def _logit_rows(s, size=4096):
    """Logits (fp32) of `size` rows at a time, with the rows' places."""
    w = s["weight"].float().t()
    for r in range(0, s["hidden"].shape[0], size):
        at = slice(r, r + size)
        yield at, torch.matmul(s["hidden"][at].float(), w).mul_(s["scale"])


def _run_plain(s):
    c = s["case"]
    if c["op"] == "loss":
        loss, lse = [], []
        for at, z in _logit_rows(s):
            t = s["target"][at].long()
            zt = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
            top = z.amax(-1, keepdim=True)
            e = z.sub_(top).exp_().sum(-1).log() + top[:, 0]
            lse.append(e)
            loss.append(torch.where(t >= 0, e - zt + c["z"] * e * e, 0.0))
        return {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    if c["op"] == "grad":
        dh, dw, w = [], 0, s["weight"].float()
        for at, z in _logit_rows(s):
            t, e = s["target"][at].long(), s["lse"][at][:, None]
            g = torch.full_like(e, s["grad_scale"])
            if s["dloss"] is not None:
                g = g * s["dloss"][at][:, None]
            g = torch.where((t >= 0)[:, None], g, 0.0)
            p = z.sub_(e).exp_().mul_(g * (1.0 + 2.0 * c["z"] * e))
            p.scatter_add_(1, t.clamp(min=0)[:, None], -g)
            dh.append(torch.matmul(p, w).mul_(s["scale"]))
            dw = dw + torch.matmul(p.t(), s["hidden"][at].float())
        return {"dhidden": torch.cat(dh).to(torch.bfloat16),
                "dweight": (dw * s["scale"]).to(torch.bfloat16)}
    if c["op"] == "tree_plan":
        return _tree_plan_plain(s, c)
    return _tree_attn_plain(s, c)


def _tree_plan_plain(s, c):
    m, words = c["q_hi"], s["mask"].shape[1]
    cu = s["cu"].long()
    lq = cu[1:] - cu[:-1]
    j = torch.arange(m, device="cuda")
    at = (cu[:-1, None] + j[None]).clamp(max=s["parents"].numel() - 1)
    up = torch.where(j[None] < lq[:, None], s["parents"][at].long(), -1)  # [n, m]
    up = torch.where(up < 0, m, up)  # m: before the tree
    up = torch.cat([up, torch.full_like(up[:, :1], m)], 1)
    seen = torch.eye(m + 1, dtype=torch.bool, device="cuda")[None].expand(c["n"], -1, -1)
    far = 1
    while far < m:  # paths of twice the length at a time
        seen = seen | torch.gather(seen, 1, up[:, :, None].expand(-1, -1, m + 1))
        up = torch.gather(up, 1, up)
        far *= 2
    seen = (seen | torch.gather(seen, 1, up[:, :, None].expand(-1, -1, m + 1)))[:, :m, :m]
    depth = seen.sum(-1) - 1
    bits = torch.nn.functional.pad(seen, (0, 32 * words - m)).view(c["n"], m, words, 32).long()
    mask = (bits << torch.arange(32, device="cuda")).sum(-1)
    mask = torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).int()
    t = torch.arange(s["parents"].numel(), device="cuda")
    i = torch.searchsorted(cu, t, right=True) - 1
    real = i < c["n"]
    i = i.clamp(max=c["n"] - 1)
    k = (t - cu[i]).clamp(max=m - 1)
    pos = torch.where(real, s["lk"][i] - lq[i] + depth[i, k], 0)
    return {"positions": pos.int(), "mask": torch.where(real[:, None], mask[i, k], 0).int()}


def _tree_attn_plain(s, c):
    n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
    group, mq, mk = hq // hkv, s["max_q"], s["max_k"]
    cu, lk = s["cu"].long(), s["lk"].long()
    lq = cu[1:] - cu[:-1]
    j = torch.arange(mq, device="cuda")
    row = (cu[:-1, None] + j[None]).clamp(max=s["q"].shape[0] - 1)
    kpos = torch.arange(mk, device="cuda")[None]
    ctx = (lk - lq)[:, None]
    table = s["table"].long()
    k = s["kc"][table].flatten(1, 2)[:, :mk].float().permute(0, 2, 3, 1)
    v = s["vc"][table].flatten(1, 2)[:, :mk].float().transpose(1, 2)
    q = s["q"][row].float().view(n, mq, hkv, group, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(n, hkv, group * mq, d), k).view(n, hkv, group, mq, mk)
    x = x.mul_(c["scale"])
    # a cached key lies at its index, a node's key at the node's position
    node = (kpos - ctx).clamp(0, mq - 1)  # [n, mk]
    where = s["positions"].long()[row]    # [n, mq]
    key_at = torch.where(kpos < ctx, kpos, torch.gather(where, 1, node))
    delta = key_at[:, None] - where[:, :, None]
    if s["bias"] is not None:
        bucket = torch.bucketize((-delta).clamp(min=0), s["edges"], right=True)
        x += s["bias"].t()[:, bucket].view(hkv, group, n, mq, mk).permute(2, 0, 1, 3, 4)
    if s["slopes"] is not None:
        x -= s["slopes"].view(1, hkv, group, 1, 1) * delta.abs().float().view(n, 1, 1, mq, mk)
    word = torch.gather(s["mask"].long()[row], 2, (node >> 5)[:, None].expand(-1, mq, -1))
    bit = ((word >> (node & 31)[:, None]) & 1).bool()
    hide = torch.where((kpos < ctx)[:, None], False, ~bit) | (kpos >= lk[:, None])[:, None]
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
# the definitions in 64 bits
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


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] in ("loss", "grad"):
        return _head_exact(s, c)
    new, ctx = _tree_lengths(c)
    ctx = _contexts(c, ctx, seed)
    parents = _trees(new, c["reach"], int(seed))
    depth, pairs = _paths(parents, new)
    if c["op"] == "tree_plan":
        pad = np.zeros(c["pad"], np.int64)
        pos = np.concatenate([np.repeat(ctx, new) + depth, pad]).astype(np.int32)
        mask = _words(pairs, s["mask"].shape[1])
        return {"positions": pos,
                "mask": np.concatenate([mask, np.zeros((c["pad"], mask.shape[1]), np.int32)])}
    return _tree_attn_exact(s, c, new, ctx, depth, pairs)


def _head_exact(s, c):
    h, w, t = s["hidden"].double(), s["weight"].double(), s["target"].long()
    loss, lse, dh = [], [], []
    dw = torch.zeros_like(w) if c["op"] == "grad" else None
    for r in range(0, c["rows"], 2048):
        z = s["scale"] * (h[r:r + 2048] @ w.t())
        e = torch.logsumexp(z, dim=1)
        tt = t[r:r + 2048]
        rows = torch.nonzero(tt >= 0)[:, 0]
        if c["op"] == "loss":
            at = torch.zeros_like(e)
            at[rows] = e[rows] - z[rows, tt[rows]] + c["z"] * e[rows] ** 2
            loss.append(at)
            lse.append(e)
            continue
        g = torch.zeros_like(e)
        g[rows] = s["grad_scale"]
        if s["dloss"] is not None:
            g = g * s["dloss"][r:r + 2048].double()
        dz = torch.softmax(z, dim=1) * (g * (1 + 2 * c["z"] * e))[:, None]
        dz[rows, tt[rows]] -= g[rows]
        dh.append(s["scale"] * (dz @ w))
        dw += s["scale"] * (dz.t() @ h[r:r + 2048])
    if c["op"] == "loss":
        return {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    return {"dhidden": torch.cat(dh), "dweight": dw}


def _tree_attn_exact(s, c, new, ctx, depth, pairs):
    hq, group = c["hq"], c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((hq, s["q"].shape[0]), float("-inf"), dtype=torch.float64, device="cuda")
    by_distance = None
    if s["bias"] is not None:
        ids = [_bucket_exact(n, c["buckets"], c["distance"]) for n in range(c["distance"] + 1)]
        by_distance = s["bias"].double()[torch.tensor(ids, device="cuda")]  # [distance, hq]
    at = 0
    for i in range(c["n"]):
        lq, lc = int(new[i]), int(ctx[i])
        lk = lc + lq
        pages = s["table"][i, :-(-lk // c["page"])].long()
        keys = s["kc"][pages].flatten(0, 1)[:lk].double()
        values = s["vc"][pages].flatten(0, 1)[:lk].double()
        see = np.zeros((lq, lk), bool)
        see[:, :lc] = True
        for j in range(lq):
            see[j, [lc + a for a in pairs[at + j]]] = True
        see = torch.as_tensor(see, device="cuda")
        d = depth[at:at + lq]
        place = torch.as_tensor(np.concatenate([np.arange(lc), lc + d]), device="cuda")
        dist = torch.as_tensor(lc + d, device="cuda")[:, None] - place[None]
        for h in range(hq):
            x = c["scale"] * (s["q"][at:at + lq, h].double() @ keys[:, h // group].t())
            if by_distance is not None:
                x = x + by_distance[:, h][dist.clamp(0, c["distance"])]
            if s["slopes"] is not None:
                x = x - float(s["slopes"][h]) * dist.abs().double()
            x = x.masked_fill(~see, float("-inf"))
            lse[h, at:at + lq] = torch.logsumexp(x, dim=-1)
            out[at:at + lq, h] = torch.softmax(x, dim=-1) @ values[:, h // group]
        at += lq
    return {"out": out, "lse": lse}
