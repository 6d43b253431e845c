"""Cases of attention with modified scores: forward, backward and the single-token step.

The scores of a query at position i and a key at position j, in head h:

    u = scale * q_i . k_j;   with a cap:  u = cap * tanh(u / cap)
    t = u - slopes[h] * |j - i| + table[bucket(j - i)][h]

and a key is visible where i, j < n (n = the sequence's valid length), where causal asks
for j <= i or j < prefix, and where both positions belong to the same document.
"""
import math

import torch

own = False

# (head_num, size_per_head) of the repository's workloads and tests.
STRUCTURES = ((4, 32), (12, 64), (16, 64), (8, 128))


# ------------------------------------------------------------------ cases
def _case(op, dtype, nh, d, batch, seq, cap=0.0, slopes=False, buckets=0, max_distance=128, both=True, causal=False,
          prefix=False, docs=0, name=None):
    c = dict(op=op, dtype=dtype, nh=nh, d=d, batch=batch, seq=seq, cap=cap, slopes=slopes, buckets=buckets,
             max_distance=max_distance, both=both, causal=causal, prefix=prefix, docs=docs)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # One short request to an encoder with a relative position table: latency counts.
        _case("forward", "fp16", 12, 64, 1, 32, buckets=32, name="fwd-table-12x64-s32-b1"),
        # The base encoder's throughput shape, relative position table.
        _case("forward", "fp16", 12, 64, 256, 128, buckets=32, name="fwd-table-12x64-s128-b256"),
        # Packed documents in rows of 512 with capped scores, the large structure.
        _case("forward", "fp16", 16, 64, 32, 512, cap=30.0, docs=4, name="fwd-cap-docs-16x64-s512-b32"),
        # A long prompt under a prefix mask with distance slopes, an odd length.
        _case("forward", "fp16", 8, 128, 2, 4093, slopes=True, causal=True, prefix=True,
              name="fwd-slopes-prefix-8x128-s4093-b2"),
        # FP32 mode, odd length, table and cap.
        _case("forward", "fp32", 4, 32, 16, 131, cap=20.0, buckets=32, name="fwd-fp32-table-cap-4x32-s131-b16"),
        # Fine-tuning the base encoder's attention and its table at its usual length.
        _case("backward", "fp16", 12, 64, 64, 128, buckets=32, name="bwd-table-12x64-s128-b64"),
        # Training on packed documents, capped scores and a table, the large structure.
        _case("backward", "fp16", 16, 64, 8, 512, cap=30.0, buckets=32, docs=4, name="bwd-table-cap-docs-16x64-s512-b8"),
        # Long rows under a prefix mask, one-directional table, an odd length.
        _case("backward", "fp16", 8, 128, 1, 4093, buckets=32, both=False, causal=True, prefix=True,
              name="bwd-table-prefix-8x128-s4093-b1"),
        # FP32 mode, odd length.
        _case("backward", "fp32", 4, 32, 8, 131, buckets=32, slopes=True, name="bwd-fp32-table-slopes-4x32-s131-b8"),
        # One sequence generating, a short cache: latency counts.
        _case("step", "fp16", 12, 64, 1, 512, slopes=True, causal=True, name="step-slopes-12x64-c512-b1"),
        # A serving batch over caches of 4096, table and cap.
        _case("step", "fp16", 16, 64, 32, 4096, cap=30.0, buckets=32, both=False, causal=True,
              name="step-table-cap-16x64-c4096-b32"),
        # FP32 mode, an odd capacity.
        _case("step", "fp32", 8, 128, 3, 1537, buckets=32, both=False, causal=True, name="step-fp32-table-8x128-c1537-b3"),
    ]


# Most pair work (batch * heads * seq^2 * size) of a drawn case of each operator, and most cache elements of a
# drawn step: those of the largest listed ones.
MOST_PAIRS = {("forward", "fp16"): 2 * 8 * 4093 ** 2 * 128, ("backward", "fp16"): 8 * 4093 ** 2 * 128,
              ("forward", "fp32"): 32 * 8 * 512 ** 2 * 64, ("backward", "fp32"): 16 * 8 * 512 ** 2 * 64}
MOST_CACHE = 32 * 16 * 4096 * 64


def draw(rng):
    op = rng.choice(("forward", "forward", "backward", "backward", "step"))
    dtype = rng.choice(("fp16", "fp16", "fp16", "fp32"))
    nh, d = rng.choice(STRUCTURES)
    low = {"forward": 1, "backward": 16, "step": 1}[op]       # one position has no gradient of its scores
    high = 512 if dtype == "fp32" and op != "step" else 4096
    seq = max(low, min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))
    if op == "step":
        most = MOST_CACHE // (nh * d * seq)
    else:
        most = MOST_PAIRS[op, dtype] // (nh * d * max(seq, 64) ** 2)
    most = max(1, min(256, most))
    batch = max(1, min(most, int(math.exp(rng.uniform(0.0, math.log(most + 1))))))
    kind = rng.choice(("table", "table", "slopes", "cap", "docs", "prefix"))
    causal = op == "step" or kind == "prefix" or rng.random() < 0.25
    return _case(op, dtype, nh, d, batch, seq,
                 cap=rng.choice((10.0, 20.0, 30.0, 50.0)) if kind == "cap" or rng.random() < 0.25 else 0.0,
                 slopes=kind == "slopes" or rng.random() < 0.15,
                 buckets=rng.choice((16, 32, 64)) if kind == "table" or rng.random() < 0.25 else 0,
                 max_distance=rng.choice((64, 128, 250, 512)), both=not causal or rng.random() < 0.25, causal=causal,
                 prefix=op != "step" and causal and (kind == "prefix" or rng.random() < 0.25),
                 docs=rng.choice((2, 4, 7)) if kind == "docs" or rng.random() < 0.2 else 0)


# ------------------------------------------------------------------ inputs
_encoders = {}


def _encoder(nh, d, dtype):
    """A handle of that structure (one layer with a small FFN; only its attention steps are called)."""
    if (nh, d, dtype) not in _encoders:
        import numpy as np
        from transformer_encoder_bert_b200 import Encoder
        h, f = nh * d, 8
        shapes = dict(w_qkv=(h, 3 * h), b_qkv=(3 * h,), w_o=(h, h), b_o=(h,), ln1_g=(h,), ln1_b=(h,), w_ff1=(h, f),
                      b_ff1=(f,), w_ff2=(f, h), b_ff2=(h,), ln2_g=(h,), ln2_b=(h,))
        t = np.float16 if dtype == "fp16" else np.float32
        _encoders[nh, d, dtype] = Encoder(nh, d, f, [{k: np.zeros(s, t) for k, s in shapes.items()}], dtype)
    return _encoders[nh, d, dtype]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    b, s, nh, d, op = case["batch"], case["seq"], case["nh"], case["d"], case["op"]
    dt = torch.float16 if case["dtype"] == "fp16" else torch.float32
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    whole = lambda low, high, *shape: torch.randint(low, high, shape, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    st = dict(case=case, batch=b, seq=s, scale=1.0 / math.sqrt(d))
    qkv = normal(3, b, nh, 1 if op == "step" else s, d)
    if case["cap"]:
        qkv[0] *= 3.0                                         # scores that reach into the cap
    st["qkv"] = qkv.to(dt)
    st["slopes"] = torch.exp2(-8.0 * torch.arange(1, nh + 1, device="cuda", dtype=torch.float32) / nh) if case["slopes"] else None
    st["table"] = normal(case["buckets"], nh) if case["buckets"] else None
    st["docs"] = None
    if case["docs"]:                                          # about that many documents to a row
        starts = torch.rand((b, s), generator=g, device="cuda") < (case["docs"] - 1) / s
        st["docs"] = starts.to(torch.int32).cumsum(1, dtype=torch.int32).contiguous()
    st["prefix"] = whole(0, s // 2 + 1, b) if case["prefix"] else None
    if op == "step":
        st["cache"] = normal(2, b, nh, s, d).to(dt)
        st["length"] = whole(s // 2, s, b)                    # tokens held: at least half of the cache
        st["ctx"] = torch.empty(b, nh * d, device="cuda", dtype=dt)
    else:
        st["valid"] = whole((s + 1) // 2, s + 1, b)
        st["ctx"] = torch.empty(b * s, nh * d, device="cuda", dtype=dt)
        st["lse"] = torch.empty(b, nh, s, device="cuda", dtype=torch.float32)
    if op == "backward":                                      # the forward's outputs, and the gradient of one of them
        out, st["lse"] = _forward(st)
        st["ctx"] = out.to(dt)
        st["dctx"] = normal(b * s, nh * d).to(dt)
        st["dqkv"] = torch.empty_like(st["qkv"])
        st["dtable"] = torch.empty_like(st["table"]) if case["buckets"] else None
    if own:
        from transformer_encoder_bert_b200 import Scores
        st["enc"] = _encoder(nh, d, case["dtype"])
        st["scores"] = Scores(scale=st["scale"], cap=case["cap"], slopes=st["slopes"], table=st["table"],
                              max_distance=case["max_distance"], bidirectional=case["both"], causal=case["causal"],
                              prefix_len=st["prefix"], doc_ids=st["docs"])
    return st


# ------------------------------------------------------------------ the plain form
def _bucket(rel, case):
    """Bucket of the relative position rel = key - query; the logarithm in 64 bits."""
    nb = case["buckets"] // 2 if case["both"] else case["buckets"]
    dist = rel.abs() if case["both"] else (-rel).clamp(min=0)
    exact = nb // 2
    far = torch.log(dist.clamp(min=1).double() / exact) / math.log(case["max_distance"] / exact) * (nb - exact)
    far = (exact + torch.floor(far + 1e-9).long()).clamp(max=nb - 1)
    return torch.where(dist < exact, dist, far) + (nb * (rel > 0) if case["both"] else 0)


def _scores(st, q, k, qpos, kpos):
    """u (after the cap), t = u + biases and key - query, of positions qpos [.., Sq, 1] and kpos [.., 1, Sk]; in 32 bits."""
    case = st["case"]
    u = torch.matmul(q.float(), k.float().transpose(-1, -2)) * st["scale"]
    if case["cap"]:
        u = case["cap"] * torch.tanh(u / case["cap"])
    rel, t = kpos - qpos, u
    if st["slopes"] is not None:
        t = t - (rel.abs().float()[..., None] * st["slopes"]).movedim(-1, -3)
    if st["table"] is not None:
        t = t + st["table"][_bucket(rel, case)].movedim(-1, -3)
    return u, t, rel


def _visible(st):
    """[batch, 1, seq, seq]: which keys a query sees."""
    s, pos = st["seq"], torch.arange(st["seq"], device="cuda")
    ok = (pos < st["valid"][:, None])
    see = ok[:, :, None] & ok[:, None, :]
    if st["case"]["causal"]:
        before = pos[None, None, :] <= pos[None, :, None]
        if st["prefix"] is not None:
            before = before | (pos[None, None, :] < st["prefix"][:, None, None])
        see = see & before
    if st["docs"] is not None:
        see = see & (st["docs"][:, :, None] == st["docs"][:, None, :])
    return see[:, None]


def _softmax(t, see):
    """exp(t - row maximum), its sum and the maximum; rows that see nothing: zeros, and a sum of 0."""
    t = torch.where(see, t, -math.inf)
    top = t.amax(-1, keepdim=True)
    e = torch.exp(t - torch.where(top > -math.inf, top, 0.0))
    return e, e.sum(-1, keepdim=True), top


def _forward(st):
    b, s, nh, d = st["batch"], st["seq"], st["case"]["nh"], st["case"]["d"]
    q, k, v = st["qkv"].unbind(0)
    pos = torch.arange(s, device="cuda")
    _, t, _ = _scores(st, q, k, pos[:, None], pos[None, :])
    e, total, top = _softmax(t, _visible(st))
    out = torch.matmul(e, v.float()) / torch.where(total > 0, total, 1.0)
    return out.transpose(1, 2).reshape(b * s, nh * d), (top + torch.log(total)).squeeze(-1)


def _backward(st):
    b, s, nh, d, case = st["batch"], st["seq"], st["case"]["nh"], st["case"]["d"], st["case"]
    q, k, v = st["qkv"].unbind(0)
    pos = torch.arange(s, device="cuda")
    u, t, rel = _scores(st, q, k, pos[:, None], pos[None, :])
    lse = st["lse"][..., None]
    p = torch.where(_visible(st), torch.exp(t - torch.where(lse > -math.inf, lse, 0.0)), 0.0)
    heads = lambda x: x.float().view(b, s, nh, d).transpose(1, 2)  # noqa: E731
    do, o = heads(st["dctx"]), heads(st["ctx"])
    dt = p * (torch.matmul(do, v.float().transpose(-1, -2)) - (do * o).sum(-1, keepdim=True))
    grads = []
    if case["buckets"]:
        by = torch.zeros(case["buckets"], nh, device="cuda", dtype=torch.float64)
        by.index_add_(0, _bucket(rel, case).reshape(-1), dt.sum(0, dtype=torch.float64).reshape(nh, -1).t())
        grads = [by.float()]
    du = dt * st["scale"]
    if case["cap"]:
        du = du * (1.0 - (u / case["cap"]) ** 2)
    dq, dk = torch.matmul(du, k.float()), torch.matmul(du.transpose(-1, -2), q.float())
    dv = torch.matmul(p.transpose(-1, -2), do)
    return [torch.stack((dq, dk, dv)).to(st["qkv"].dtype)] + grads


def _step(st):
    b, nh, d, cache = st["batch"], st["case"]["nh"], st["case"]["d"], st["cache"]
    at, rows = st["length"].long(), torch.arange(b, device="cuda")
    cache[:, rows, :, at] = st["qkv"][1:, :, :, 0].transpose(0, 1)
    pos = torch.arange(st["seq"], device="cuda")
    _, t, _ = _scores(st, st["qkv"][0], cache[0], at[:, None, None], pos[None, None, :])
    see = pos <= at[:, None]
    if st["docs"] is not None:
        see = see & (st["docs"] == st["docs"].gather(1, at[:, None]))
    e, total, _ = _softmax(t, see[:, None, None, :])
    return (torch.matmul(e, cache[1].float()) / total).reshape(b, nh * d).to(cache.dtype)


def run(st):
    case = st["case"]
    if own:
        enc, sc, b, s = st["enc"], st["scores"], st["batch"], st["seq"]
        if case["op"] == "forward":
            enc.op_scored_attention(sc, st["qkv"], st["valid"], st["ctx"], b, s, lse=st["lse"])
            return [st["ctx"], st["lse"]]
        if case["op"] == "backward":
            enc.op_scored_attention_backward(sc, st["qkv"], st["valid"], st["ctx"], st["lse"], st["dctx"], st["dqkv"], b, s,
                                             dtable=st["dtable"])
            return [st["dqkv"]] + ([st["dtable"]] if case["buckets"] else [])
        enc.op_scored_attention_step(sc, st["qkv"], st["cache"], st["length"], st["ctx"], b, s)
        return [st["ctx"], st["cache"]]
    if case["op"] == "forward":
        out, lse = _forward(st)
        return [out.to(st["qkv"].dtype), lse]
    if case["op"] == "backward":
        return _backward(st)
    return [_step(st), st["cache"]]


# ------------------------------------------------------------------ work and the 64-bit definition
def work(case):
    """Means over the lengths that prepare draws (n in [S/2, S]; documents of n / docs on average)."""
    b, s, nh, d = case["batch"], case["seq"], case["nh"], case["d"]
    e = 2 if case["dtype"] == "fp16" else 4
    n, h = 0.75 * s, nh * d
    if case["op"] == "step":
        keys = (n + 0.5) / (2 if case["docs"] else 1)
        return {"bytes": b * e * (2 * (n + 1) * h + 6 * h), "flops": 4.0 * b * nh * keys * d}
    pairs = (7 / 12) * s * s
    if case["docs"]:
        pairs *= 2 / (case["docs"] + 1)
    if case["causal"]:
        pairs *= 0.62 if case["prefix"] else 0.5
    pairs *= b * nh
    if case["op"] == "forward":
        return {"bytes": 3 * b * n * h * e + b * s * (h * e + 4 * nh), "flops": 4.0 * pairs * d}
    return {"bytes": b * n * (5 * h * e + 4 * nh) + 3 * b * s * h * e, "flops": 10.0 * pairs * d}


def exact(case, seed):
    st = prepare(case, seed)
    b, s, nh, d = case["batch"], case["seq"], case["nh"], case["d"]
    f8 = torch.float64
    pos = torch.arange(s, device="cuda")
    count = case["buckets"] // 2 if case["both"] else case["buckets"]

    def bucket_of(r):                                         # r: key - query, one integer
        a = abs(r) if case["both"] else max(-r, 0)
        c = a
        if a >= count // 2:
            f = math.log(a / (count // 2)) / math.log(case["max_distance"] / (count // 2)) * (count - count // 2)
            c = min(count - 1, count // 2 + math.floor(f + 1e-9))
        return c + (count if case["both"] and r > 0 else 0)

    buckets = torch.tensor([bucket_of(r) for r in range(1 - s, s)], device="cuda") if case["buckets"] else None
    valid = (st["length"] + 1 if case["op"] == "step" else st["valid"]).tolist()
    prefix = st["prefix"].tolist() if st["prefix"] is not None else [0] * b
    qkv = st["qkv"]
    if case["op"] == "step":
        cache = st["cache"].clone()
        for i in range(b):
            cache[0, i, :, valid[i] - 1] = qkv[1, i, :, 0]
            cache[1, i, :, valid[i] - 1] = qkv[2, i, :, 0]
        ctx = torch.zeros(b, nh, d, device="cuda", dtype=f8)
    else:
        ctx = torch.zeros(b, s, nh, d, device="cuda", dtype=f8)
        lse = torch.full((b, nh, s), -math.inf, device="cuda", dtype=f8)
        grad = torch.zeros(3, b, nh, s, d, device="cuda", dtype=f8)
        by = torch.zeros(max(1, case["buckets"]), nh, device="cuda", dtype=f8)
    for i in range(b):
        n = valid[i]
        first = n - 1 if case["op"] == "step" else 0
        rel = pos[None, :n] - pos[first:n, None]
        hide = torch.zeros_like(rel, dtype=torch.bool)
        if case["causal"]:
            hide = (rel > 0) & (pos[None, :n] >= prefix[i])
        if st["docs"] is not None:
            hide = hide | (st["docs"][i, None, :n] != st["docs"][i, first:n, None])
        for h in range(nh):
            if case["op"] == "step":
                q, k, v = qkv[0, i, h].to(f8), cache[0, i, h, :n].to(f8), cache[1, i, h, :n].to(f8)
            else:
                q, k, v = (qkv[x, i, h, :n].to(f8) for x in range(3))
            raw = q @ k.T * st["scale"]
            slope = 1.0
            if case["cap"]:
                th = torch.tanh(raw / case["cap"])
                raw, slope = case["cap"] * th, 1 - th * th
            if st["slopes"] is not None:
                raw = raw - st["slopes"][h].to(f8) * rel.abs()
            if buckets is not None:
                raw = raw + st["table"][:, h].to(f8)[buckets[rel + s - 1]]
            raw = raw.masked_fill(hide, -math.inf)
            if case["op"] == "backward":
                p = torch.exp(raw - st["lse"][i, h, :n, None].to(f8)).masked_fill(hide, 0.0)
                do = st["dctx"].view(b, s, nh, d)[i, :n, h].to(f8)
                o = st["ctx"].view(b, s, nh, d)[i, :n, h].to(f8)
                g = p * (do @ v.T - (do * o).sum(1, keepdim=True))
                if buckets is not None:
                    by[:, h].index_add_(0, buckets[rel + s - 1].reshape(-1), g.reshape(-1))
                g = g * slope * st["scale"]
                grad[0, i, h, :n], grad[1, i, h, :n], grad[2, i, h, :n] = g @ k, g.T @ q, p.T @ do
            else:
                z = torch.logsumexp(raw, 1)
                o = torch.exp(raw - z[:, None]) @ v
                if case["op"] == "step":
                    ctx[i, h] = o[0]
                else:
                    ctx[i, :n, h], lse[i, h, :n] = o, z
    if case["op"] == "backward":
        return [grad] + ([by] if case["buckets"] else [])
    if case["op"] == "step":
        return [ctx.reshape(b, nh * d), None]
    return [ctx.reshape(b * s, nh * d), lse]
