"""Attention with modified scores at the ends of its ranges: every form of the cap, the largest
tables, documents of any id, buffers whose offsets pass 2^31 elements, sequences of 65536, and
calls on another stream, in a graph, and without programmatic dependent launch.

Tolerances: check_forward and check_backward of test_gpu_scored (bounds from the arithmetic), or
equality where the same arithmetic must give the same bits.
"""
import numpy as np
import pytest
import torch

import encoder_inputs as EI
from oracle import scored_oracle as SO
from parity_utils import encoder_from_inputs, to_dev
from test_gpu_scored import Case, _formats, check_backward, check_forward, encoder, handle
from transformer_encoder_bert_b200 import EncError, Scores

pytestmark = pytest.mark.gpu


# (scale, cap, factor of q): |scale q.k / cap| of q, k ~ N(0, 1), d = 64 is at most about
# 45 factor scale / cap.
@pytest.mark.parametrize("scale,cap,factor", [
    (0.125, 30.0, 1.0),            # all below 0.5
    (0.125, 8.0, 1.0),             # some blocks above 0.5, none above 1.25
    (0.125, 3.0, 1.0),             # around 1.25
    (0.125, 0.25, 1.0),            # mostly far above
    (-0.125, 20.0, 1.0),           # a negative scale
    (5e-3, 1e4, 8.0),              # a ratio of scale to cap too small to be folded into coefficients
    (2.0, 1e-3, 0.01),             # a large one
    (20.0, 1e-3, 0.01),            # one too large to be folded
], ids=str)
@pytest.mark.parametrize("nh,d,s", [(4, 32, 300), (3, 64, 90), (3, 64, 300), (2, 128, 128), (2, 128, 300)], ids=str)
def test_every_form_of_the_cap(nh, d, s, scale, cap, factor):
    c = Case("table", "fp16", 2, nh, s, d, seed=7)
    c.spec.scale, c.spec.cap = float(np.float32(scale)), float(np.float32(cap))
    c.qkv[0] = (c.qkv[0] * factor).astype(np.float16)
    ctx, lse = c.forward()
    check_forward(c, ctx, lse)
    check_backward(c, ctx, lse, *c.backward(ctx, lse))


@pytest.mark.parametrize("nh,d,s", [(4, 32, 260), (3, 64, 100), (3, 64, 260), (2, 128, 260)], ids=str)
def test_forms_of_the_cap_in_one_call(nh, d, s):
    """Queries that grow along the sequence: warps of one tile take different forms."""
    c = Case("cap-docs", "fp16", 2, nh, s, d, seed=8)
    c.qkv[0] = (c.qkv[0] * np.geomspace(0.02, 4, s)[None, None, :, None]).astype(np.float16)
    ctx, lse = c.forward()
    check_forward(c, ctx, lse)
    check_backward(c, ctx, lse, *c.backward(ctx, lse))


@pytest.mark.parametrize("mode,nh,d", [("fp16", 3, 64), ("fp16", 2, 128), ("fp32", 4, 32)])
def test_largest_table(mode, nh, d):
    s = 1100
    c = Case("prefix", mode, 1, nh, s, d, seed=9, valid=[1090])
    c.spec.table = np.random.default_rng(1).standard_normal((128, nh)).astype(np.float32)
    c.spec.max_distance, c.spec.bidirectional = 2048, True
    ctx, lse = c.forward()
    check_forward(c, ctx, lse)
    check_backward(c, ctx, lse, *c.backward(ctx, lse))


@pytest.mark.parametrize("mode", ["fp16", "fp32"])
@pytest.mark.parametrize("s", [100, 300])
@pytest.mark.parametrize("kind", ["each its own", "interleaved", "extremes"])
def test_documents_of_any_id(kind, s, mode):
    c = Case("plain", mode, 2, 3, s, 64, seed=10, valid=[s, s - 37])
    top, low = np.iinfo(np.int32).max, np.iinfo(np.int32).min
    c.spec.doc_ids = {
        "each its own": np.tile(np.arange(s)[::-1], (2, 1)),
        "interleaved": np.tile(np.arange(s) % 3, (2, 1)),
        "extremes": np.where(np.arange(s)[None] < np.array([[s // 3], [70]]), low, np.where(np.arange(s) % 5 == 0, 0, top)),
    }[kind].astype(np.int32)
    ctx, lse = c.forward()
    check_forward(c, ctx, lse)
    check_backward(c, ctx, lse, *c.backward(ctx, lse))


@pytest.mark.parametrize("mode", ["fp16", "fp32"])
@pytest.mark.parametrize("s", [100, 300])
def test_without_dependent_launch(s, mode):
    c = Case("cap-slopes-table-prefix-docs", mode, 3, 3, s, 64, seed=11)
    ctx, lse = c.forward()
    want = c.backward(ctx, lse)
    enc = encoder(3, 64, mode)
    enc.set_option("pdl", False)
    try:
        again, lse2 = c.forward()
        got = c.backward(again, lse2)
    finally:
        enc.set_option("pdl", True)
    assert torch.equal(ctx, again) and torch.equal(lse, lse2)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("mode", ["fp16", "fp32"])
def test_backward_and_step_on_another_stream(mode):
    c = Case("table", mode, 2, 3, 200, 64, seed=12)
    ctx, lse = c.forward()
    want = c.backward(ctx, lse)
    enc = encoder(3, 64, mode)
    sc, qkv, vl, dctx = c.scores(), to_dev(c.qkv), to_dev(c.valid), to_dev(c.dctx).view(c.b * c.s, -1)
    dqkv, dtable = torch.empty_like(qkv), torch.empty_like(want[1])
    new = qkv[:, :, :, :1].contiguous()
    cache, length = qkv[1:].clone(), torch.tensor([150, 199], dtype=torch.int32, device="cuda")
    out, out2 = (torch.empty((2, 192), dtype=qkv.dtype, device="cuda") for _ in range(2))
    cache2 = cache.clone()
    enc.op_scored_attention_step(sc, new, cache2, length, out2, 2, 200)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    enc.op_scored_attention_backward(sc, qkv, vl, ctx, lse, dctx, dqkv, 2, 200, dtable=dtable, stream=side)
    enc.op_scored_attention_step(sc, new, cache, length, out, 2, 200, stream=side)
    side.synchronize()
    assert torch.equal(dqkv, want[0]) and torch.equal(dtable, want[1])
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(cache, cache2)


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
def test_captured_steps_follow_the_lengths(dtype):
    """A step captured once and replayed for a run of tokens: positions come from len on the device."""
    nh, d, cap, b = 3, 64, 40, 2
    c = Case("table-one-way-causal", dtype, b, nh, cap, d, seed=13, valid=[cap] * b)
    enc, sc = encoder(nh, d, dtype), c.scores()
    tokens = to_dev(c.qkv)
    new, out = tokens[:, :, :, :1].contiguous(), torch.empty((b, nh * d), dtype=tokens.dtype, device="cuda")
    cache = torch.zeros((2, b, nh, cap, d), dtype=tokens.dtype, device="cuda")
    length = torch.tensor([0, 7], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        g.capture_begin(capture_error_mode="thread_local")
        enc.op_scored_attention_step(sc, new, cache, length, out, b, cap)
        g.capture_end()
    torch.cuda.synchronize()
    cache2, length2, out2 = cache.clone(), length.clone(), torch.empty_like(out)
    for p in range(cap):                                      # the second sequence runs out of room at 33
        new.copy_(tokens[:, :, :, p : p + 1])
        g.replay()
        enc.op_scored_attention_step(sc, new, cache2, length2, out2, b, cap)
        assert torch.equal(out, out2)
        length += 1
        length2 += 1
    assert torch.equal(cache, cache2)
    assert torch.equal(cache[:, 0], tokens[1:, 0]) and torch.equal(cache[:, 1, :, 7:], tokens[1:, 1, :, : cap - 7])
    assert (out[1] == 0).all()


def _big_sequence(mode, nh, d, s, b):
    """One full sequence behind b - 1 short ones: its rows are the same as by itself."""
    c = Case("cap-slopes", mode, 1, nh, s, d, seed=14)
    enc, sc = encoder(nh, d, mode), c.scores()
    ctx, lse = c.forward()
    dqkv, _ = c.backward(ctx, lse)
    qkv = torch.zeros((3, b, nh, s, d), dtype=dqkv.dtype, device="cuda")
    dctx = torch.zeros((b, s, nh * d), dtype=dqkv.dtype, device="cuda")
    assert qkv.numel() > 2 ** 31
    qkv[:, -1] = to_dev(c.qkv)[:, 0]
    dctx[-1] = to_dev(c.dctx).view(s, -1)
    valid = torch.ones(b, dtype=torch.int32, device="cuda")
    valid[-1] = s
    out = torch.empty((b * s, nh * d), dtype=dqkv.dtype, device="cuda")
    lse2 = torch.empty((b, nh, s), device="cuda")
    enc.op_scored_attention(sc, qkv, valid, out, b, s, lse=lse2)
    assert torch.equal(out[-s:], ctx) and torch.equal(lse2[-1], lse[0])
    assert (out[: (b - 1) * s] == 0).all() and (lse2[:-1, :, 0] == 0).all() and torch.isneginf(lse2[:-1, :, 1:]).all()
    grad = torch.empty_like(qkv)
    enc.op_scored_attention_backward(sc, qkv, valid, out, lse2, dctx.view(b * s, -1), grad, b, s)
    assert enc.device_status() == 0
    assert torch.equal(grad[:, -1], dqkv[:, 0])
    assert not grad[:, :-1].any()


@pytest.mark.parametrize("mode,nh,d,s,b", [("fp16", 4, 32, 128, 65535), ("fp16", 3, 64, 300, 13000),
                                           ("fp16", 2, 128, 300, 10000), ("fp32", 4, 32, 100, 65535)], ids=str)
def test_buffers_past_2_31_elements(mode, nh, d, s, b):
    try:
        _big_sequence(mode, nh, d, s, b)
    finally:
        torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
def test_step_over_a_cache_past_2_31_elements(dtype):
    nh, d, cap, b = 2, 128, 65536, 130
    r = np.random.default_rng(15)
    np_dt = np.float16 if dtype == "fp16" else np.float32
    held = r.standard_normal((2, nh, cap, d)).astype(np_dt)
    new = r.standard_normal((3, b, nh, 1, d)).astype(np_dt)
    length = np.zeros(b, np.int32)
    length[-1] = cap - 1
    try:
        cache = torch.zeros((2, b, nh, cap, d), dtype=to_dev(new).dtype, device="cuda")
        assert cache[0].numel() > 2 ** 31
        cache[:, -1] = to_dev(held)
        ctx = torch.empty((b, nh * d), dtype=cache.dtype, device="cuda")
        slopes = np.full(nh, 2.0 ** -12, np.float32)
        enc = handle(nh, d, dtype)
        enc.op_scored_attention_step(Scores(slopes=to_dev(slopes)), to_dev(new), cache, to_dev(length), ctx, b, cap)
        got = ctx.cpu().numpy().astype(np.float64).reshape(b, nh, d)
        assert np.array_equal(cache[:, :, :, 0].cpu().numpy()[:, :-1], new[1:, :-1, :, 0])
        assert np.array_equal(cache[:, -1, :, -1].cpu().numpy(), new[1:, -1, :, 0])
        assert not cache[:, :-1, :, 1:].any()
        assert torch.equal(cache[:, -1, :, :-1], to_dev(held[:, :, :-1]))
    finally:
        cache = None
        torch.cuda.empty_cache()
    _, eps_out, tiny = _formats(dtype)
    assert (np.abs(got[:-1] - new[2, :-1, :, 0]) <= 2 * eps_out * np.abs(new[2, :-1, :, 0].astype(np.float64)) + tiny).all()
    held[:, :, -1] = new[1:, -1, :, 0]
    spec = SO.ScoreSpec(scale=float(np.float32(d ** -0.5)), slopes=slopes)
    ref, _ = SO.step(spec, new[:, -1:], held[:, None].copy(), length[-1:])
    dots = spec.scale * (np.abs(new[0, -1, :, 0].astype(np.float64))[:, None] @ np.swapaxes(np.abs(held[0].astype(np.float64)), 1, 2)).max()
    top = dots + 2.0 ** -12 * cap
    # t as in the tests of short caches; sums of cap terms are made of partial sums over at most cap / 128 rows a lane
    # and then over lanes, warps and CTAs, so cap + 8 roundings bound them amply.
    rel = 2 * ((d + 8) * 2.0 ** -23 * dots + 8 * 2.0 ** -24 * top) + 2.0 ** -20 + (cap + 8) * 2.0 ** -23
    p_abs = np.abs(held[1]).astype(np.float64).max()
    assert (np.abs(got[-1:] - ref.reshape(1, nh, d)) <= 2 * rel * p_abs + eps_out * np.abs(ref.reshape(1, nh, d)) + tiny).all()


@pytest.mark.parametrize("mode,nh,d", [("fp16", 3, 64), ("fp16", 2, 128), ("fp32", 4, 32)])
def test_longest_sequence(mode, nh, d):
    """65536 tokens, causal with a prefix, slopes: rows and columns here and there against 64-bit arithmetic."""
    s, prefix, n = 65536, 1000, 65500
    enc = encoder(nh, d, mode)
    g = torch.Generator(device="cuda").manual_seed(16)
    dt = torch.float16 if mode == "fp16" else torch.float32
    qkv = torch.randn((3, 1, nh, s, d), device="cuda", generator=g).to(dt)
    dctx = torch.randn((s, nh * d), device="cuda", generator=g).to(dt)
    slopes = torch.full((nh,), 2.0 ** -10, device="cuda")
    sc = Scores(slopes=slopes, causal=True, prefix_len=torch.tensor([prefix], dtype=torch.int32, device="cuda"))
    valid = torch.tensor([n], dtype=torch.int32, device="cuda")
    ctx, lse = torch.empty_like(dctx), torch.empty((1, nh, s), device="cuda")
    enc.op_scored_attention(sc, qkv, valid, ctx, 1, s, lse=lse)
    grad = torch.empty_like(qkv)
    enc.op_scored_attention_backward(sc, qkv, valid, ctx, lse, dctx, grad, 1, s)
    assert enc.device_status() == 0
    assert not ctx[n:].any() and torch.isneginf(lse[0, :, n:]).all() and not grad[:, 0, :, n:].any()
    q, k, v = (qkv[i, 0].double() for i in range(3))
    o, do = (x.view(s, nh, d).transpose(0, 1).double() for x in (ctx, dctx))
    dsum = (o * do).sum(-1)
    pos = torch.arange(s, device="cuda")
    at = torch.tensor([0, 1, 63, 64, 127, 128, 999, 1000, 1001, 5000, 32767, 32768, 40000, 65407, 65498, 65499], device="cuda")

    def see(i, j):
        return ((j <= i) | (j < prefix)) & (i < n) & (j < n)

    def scores(qi, kj, i, j):
        t = qi @ kj.transpose(-1, -2) * d ** -0.5 - 2.0 ** -10 * (i[:, None] - j[None]).abs()
        return t.masked_fill(~see(i[:, None], j[None]), float("-inf"))

    t = scores(q[:, at], k, at, pos)
    ref_lse, p = torch.logsumexp(t, -1), torch.softmax(t, -1)
    # Errors of t: d + 8 roundings of 2^-23 of sum |q| |k| scale (< 16) and 4 of 2^-24 of |t2| < 128: below 2^-11.7.
    # So P is off by less than 2^-11.6 relative, by 2^-11 more where it is a half, and D and the sums (of 32 to 64
    # partial sums' magnitude each) by far less: 2^-9 of the sums of absolute values.  Halves below 2^-14 are off by
    # 2^-25 of their scale instead: of the row's largest P in the forward (whose l is at least 1), of 1 and of dU's
    # scale in the backward.
    rel, tiny, eps = 2.0 ** -9, 2.0 ** -25, 2.0 ** -11
    assert (lse[0][:, at].double() - ref_lse).abs().max() < 2.0 ** -10
    seen = see(at[:, None], pos[None]).double()
    ref = p @ v
    assert ((o[:, at] - ref).abs() <= rel * (p @ v.abs()) + tiny * (seen @ v.abs()) + eps * ref.abs() + tiny).all()
    norm = do.norm(dim=-1).amax(-1) * v.norm(dim=-1).amax(-1)                             # of dU's scale, [nh]
    step = 2.0 ** -36 * norm[:, None, None]                                              # its smallest step, twice
    du = p * (do[:, at] @ v.transpose(-1, -2) - dsum[:, at, None])
    size = p * (do[:, at].abs() @ v.abs().transpose(-1, -2) + dsum[:, at, None].abs())
    err = d ** -0.5 * ((rel * size + step * seen) @ k.abs()) + tiny
    dq = d ** -0.5 * (du @ k)
    assert ((grad[0, 0][:, at].double() - dq).abs() <= err + eps * dq.abs()).all()
    t = scores(q, k[:, at], pos, at)
    p = torch.exp(t - lse[0].double().masked_fill(torch.isneginf(lse[0]), 0)[..., None])
    dv = p.transpose(-1, -2) @ do
    seen = see(pos[:, None], at[None]).double()
    assert ((grad[2, 0][:, at].double() - dv).abs()
            <= (rel * p + tiny * seen).transpose(-1, -2) @ do.abs() + eps * dv.abs() + tiny).all()
    du = p * (do @ v[:, at].transpose(-1, -2) - dsum[..., None])
    size = p * (do.abs() @ v[:, at].abs().transpose(-1, -2) + dsum[..., None].abs())
    dk = d ** -0.5 * (du.transpose(-1, -2) @ q)
    err = d ** -0.5 * ((rel * size + step * seen).transpose(-1, -2) @ q.abs()) + tiny
    assert ((grad[1, 0][:, at].double() - dk).abs() <= err + eps * dk.abs()).all()


def test_two_handles_at_once():
    """Handles share nothing: backward calls of two of them on two streams."""
    inp = EI.make_inputs(EI.Workload("scored", EI.EncoderShape(3, 64, 64, 1), 1, 1, "fp16", 1, 1, seed=0))
    encs, cases = [encoder_from_inputs(inp) for _ in range(2)], [Case("table", "fp16", 4, 3, 300, 64, seed=s) for s in (17, 18)]
    want, got, args = [], [], []
    for e, c in zip(encs, cases):
        ctx, lse = c.forward(e)
        want.append(c.backward(ctx, lse, e))
        args.append((c.scores(), to_dev(c.qkv), to_dev(c.valid), ctx, lse, to_dev(c.dctx).view(c.b * c.s, -1)))
        got.append((torch.empty_like(want[-1][0]), torch.empty_like(want[-1][1])))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for e, st, a, (dqkv, dtable) in zip(encs, streams, args, got):
            e.op_scored_attention_backward(*a, dqkv, 4, 300, dtable=dtable, stream=st)
    torch.cuda.synchronize()
    for w, x in zip(want, got):
        assert torch.equal(w[0], x[0]) and torch.equal(w[1], x[1])
    for e in encs:
        e.close()


def test_too_large_is_refused():
    enc, c = handle(4, 32, "fp16"), Case("plain", "fp16", 1, 4, 16, 32)
    x = to_dev(c.qkv)
    with pytest.raises((EncError, ValueError)):
        enc.op_scored_attention(c.scores(), x, to_dev(c.valid), torch.empty((16, 128), dtype=x.dtype, device="cuda"), 1, 65537)
    with pytest.raises(EncError, match="65535"):
        enc.reserve_scored(65536, 1)
