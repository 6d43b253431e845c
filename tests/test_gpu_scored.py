"""Attention with modified scores on the GPU against the float64 oracle: forward, backward,
single-token step, and the encoder forward that uses it.

Tolerances are elementwise bounds from the arithmetic (_t_error, check_forward,
check_backward): FP32 dot products of
d terms (products of halves are exact, an accumulation step is off by at most 2^-23 of its
partial sum on the tensor cores, 2^-24 on the CUDA cores), the exponential's and tanh's
approximations, one FP16 rounding (2^-11) of P or dU in FP16 mode, and one rounding of the
result.
"""
import numpy as np
import pytest
import torch

import encoder_inputs as EI
from oracle import encoder_oracle as EO
from oracle import scored_oracle as SO
from parity_utils import encoder_from_inputs, rel_l2, to_dev
from transformer_encoder_bert_b200 import EncError, Scores

pytestmark = pytest.mark.gpu

STRUCTURES = [(4, 32), (3, 64), (2, 128)]
_handles = {}


def handle(nh, d, dtype):
    if (nh, d, dtype) not in _handles:
        inp = EI.make_inputs(EI.Workload("scored", EI.EncoderShape(nh, d, 64, 1), 1, 1, dtype, 1, 1, seed=0))
        _handles[nh, d, dtype] = encoder_from_inputs(inp)
    return _handles[nh, d, dtype]


@pytest.fixture(params=["fp16", "fp16-simt", "fp32"])
def mode(request):
    return request.param


def encoder(nh, d, mode):
    enc = handle(nh, d, mode[:4])
    enc.set_option("tc_attention", mode != "fp16-simt")
    return enc


class Case:
    """Inputs of one call on both sides."""

    def __init__(self, kind, mode, b, nh, s, d, seed=0, valid=None, std=1.0):
        r = np.random.default_rng(seed + 1000)
        self.b, self.nh, self.s, self.d, self.mode = b, nh, s, d, mode
        np_dt = np.float16 if mode.startswith("fp16") else np.float32
        self.qkv = (r.standard_normal((3, b, nh, s, d)) * std).astype(np_dt)
        self.dctx = r.standard_normal((b, s, nh, d)).astype(np_dt)
        if valid is None:
            valid = r.integers(max(1, s // 2), s + 1, b)
            valid[0] = s
        self.valid = np.asarray(valid, np.int32)
        self.spec = SO.ScoreSpec(scale=float(np.float32(d ** -0.5)))
        if "cap" in kind:
            self.spec.cap = 2.5
        if "slopes" in kind:
            self.spec.slopes = (2.0 ** -np.arange(1, nh + 1)).astype(np.float32)
        if "table" in kind:
            both = "one-way" not in kind
            self.spec.table = r.standard_normal((16 if both else 10, nh)).astype(np.float32)
            self.spec.max_distance, self.spec.bidirectional = 37, both
        if "causal" in kind or "prefix" in kind:
            self.spec.causal = True
        if "prefix" in kind:
            self.spec.prefix_len = r.integers(0, s + 2, b).astype(np.int32)
        if "docs" in kind:
            self.spec.doc_ids = np.sort(r.integers(0, 4, (b, s)), 1).astype(np.int32)
        if "shuffled" in kind:
            self.spec.doc_ids = r.integers(-2, 2, (b, s)).astype(np.int32)

    def scores(self):
        sp = self.spec
        dev = lambda x: None if x is None else to_dev(x)  # noqa: E731
        return Scores(scale=sp.scale, cap=sp.cap, slopes=dev(sp.slopes), table=dev(sp.table), max_distance=sp.max_distance,
                      bidirectional=sp.bidirectional, causal=sp.causal, prefix_len=dev(sp.prefix_len),
                      doc_ids=dev(sp.doc_ids))

    def forward(self, enc=None, lse=True):
        enc = enc or encoder(self.nh, self.d, self.mode)
        qkv = to_dev(self.qkv)
        ctx = torch.full((self.b * self.s, self.nh * self.d), float("nan"), dtype=qkv.dtype, device="cuda")
        out = torch.full((self.b, self.nh, self.s), float("nan"), device="cuda") if lse else None
        enc.op_scored_attention(self.scores(), qkv, to_dev(self.valid), ctx, self.b, self.s, lse=out)
        assert enc.device_status() == 0
        return ctx, out

    def backward(self, ctx, lse, enc=None):
        enc = enc or encoder(self.nh, self.d, self.mode)
        qkv = to_dev(self.qkv)
        dqkv = torch.full(qkv.shape, float("nan"), dtype=qkv.dtype, device="cuda")
        dtable = None if self.spec.table is None else torch.full(self.spec.table.shape, float("nan"), device="cuda")
        enc.op_scored_attention_backward(self.scores(), qkv, to_dev(self.valid), ctx, lse,
                                         to_dev(self.dctx).view(self.b * self.s, -1), dqkv, self.b, self.s, dtable=dtable)
        assert enc.device_status() == 0
        return dqkv, dtable

    def shaped(self, ctx):
        return ctx.cpu().numpy().astype(np.float64).reshape(self.b, self.s, self.nh, self.d)


def _t_error(c):
    """Bound on the error of any t of the case: the dot product, its scaling, the cap, the bias, and the
    rounding of t in units of log2 (at most 4 roundings of |t| by 2^-24, twice counted).  The bounds take |scale|:
    errors of a product are relative to its magnitude, whatever the scale's sign."""
    q, k = (SO._clean(c.qkv[i], c.valid, 2) for i in range(2))
    dots = abs(c.spec.scale) * (np.abs(q) @ np.swapaxes(np.abs(k), -1, -2)).max()
    pos = np.arange(c.s)
    t, _ = SO.scores(c.spec, q, k, pos, pos)
    top = np.abs(t).max() + np.abs(SO.bias(c.spec, c.nh, pos, pos)).max() + c.spec.cap
    return (c.d + 8) * 2.0 ** -23 * dots + 8 * 2.0 ** -24 * top + c.spec.cap * 2.0 ** -20


def _formats(mode):
    """(rounding of P and dU, rounding of the result, smallest steps of both)."""
    return (2.0 ** -11, 2.0 ** -11, 2.0 ** -25) if mode.startswith("fp16") else (0.0, 2.0 ** -24, 0.0)


def check_forward(c, ctx, lse):
    eps_p, eps_out, tiny = _formats(c.mode)
    ref, ref_lse, p = SO.forward(c.spec, c.qkv, c.valid)
    v = SO._clean(c.qkv[2], c.valid, 2)
    dt = _t_error(c)
    rel = 2 * dt + 2.0 ** -20 + (c.s + 8) * 2.0 ** -23     # of P, of its sum, and of sums of c.s terms
    mass = np.swapaxes(p @ np.abs(v), 1, 2)
    bound = (eps_p + 2 * rel) * mass + eps_out * np.abs(ref) + tiny * (1 + c.s * np.abs(v).max())
    got = c.shaped(ctx)
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= bound * 1.001).all(), np.max(np.abs(got - ref) / (bound + 1e-30))
    if lse is not None:
        got = lse.cpu().numpy().astype(np.float64)
        seen = np.isfinite(ref_lse)
        assert (np.isneginf(got) == ~seen).all()
        assert (np.abs(got[seen] - ref_lse[seen]) <= dt + rel + 2.0 ** -22 * np.abs(ref_lse[seen])).all()


def check_backward(c, ctx, lse, dqkv, dtable):
    eps_p, eps_out, tiny = _formats(c.mode)
    lse = lse.cpu().numpy().astype(np.float64)
    ref, ref_table, (p, size, du) = SO.backward(c.spec, c.qkv, c.valid, c.shaped(ctx), lse, c.dctx)
    q, k, v = (np.abs(SO._clean(c.qkv[i], c.valid, 2)) for i in range(3))
    do = np.abs(np.swapaxes(SO._clean(c.dctx, c.valid, 1), 1, 2))
    rel = 2 * _t_error(c) + 2.0 ** -19 + (c.s + c.d + 8) * 2.0 ** -23
    # An FP16 value below 2^-14 of its scale is off by up to 2^-25 of it; dU's scale puts the largest
    # |dctx_i| |v_j| of the (sequence, head) at 2^13 or more, P's is 1.
    norm = np.sqrt((do ** 2).sum(-1)).max(-1) * np.sqrt((v ** 2).sum(-1)).max(-1)          # [B, nh]
    tiny_du = tiny * 2.0 ** -12 * 2 * norm[..., None, None]
    err_du = eps_p * np.abs(du) + 2 * rel * size + tiny_du
    err_p = (eps_p + 2 * rel) * p + tiny
    seen = p > 0
    err_du, err_p = np.where(seen, err_du, 0), np.where(seen, err_p, 0)
    scale = abs(c.spec.scale)
    bound = np.stack((scale * (err_du @ k), scale * (np.swapaxes(err_du, -1, -2) @ q),
                      np.swapaxes(err_p, -1, -2) @ do)) + eps_out * np.abs(ref) + tiny
    got = dqkv.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - ref) / (bound * 1.001 + 1e-30), axis=(1, 2, 3, 4))
    assert (worst <= 1).all(), worst
    for b, n in enumerate(np.clip(c.valid, 0, c.s)):
        assert (got[:, b, :, n:] == 0).all()
    if dtable is not None:
        err = np.zeros(ref_table.shape)
        pos = np.arange(c.s)
        np.add.at(err, SO.bucket_matrix(c.spec, pos, pos), np.moveaxis((2 * rel * size).sum(0), 0, -1))
        assert (np.abs(dtable.cpu().numpy() - ref_table) <= err + 2.0 ** -23 * np.abs(ref_table) + 1e-30).all()


KINDS = ["plain", "cap", "slopes", "table", "table-one-way-causal", "prefix", "docs", "shuffled",
         "cap-slopes-table-prefix-docs"]
SEQS = [1, 2, 31, 64, 65, 127, 128, 129, 200, 257, 400]


@pytest.mark.parametrize("nh,d", STRUCTURES, ids=lambda v: str(v))
@pytest.mark.parametrize("s", SEQS, ids=lambda v: f"s{v}")
@pytest.mark.parametrize("kind", KINDS)
def test_forward_and_backward(kind, s, nh, d, mode):
    c = Case(kind, mode, 3, nh, s, d, seed=s)
    ctx, lse = c.forward()
    check_forward(c, ctx, lse)
    check_backward(c, ctx, lse, *c.backward(ctx, lse))


@pytest.mark.parametrize("nh,d", STRUCTURES, ids=lambda v: str(v))
def test_lengths_of_zero_and_out_of_range(nh, d, mode):
    c = Case("table-causal", mode, 5, nh, 70, d, valid=[0, -3, 1, 70, 500])
    ctx, lse = c.forward()
    check_forward(c, ctx, lse)
    check_backward(c, ctx, lse, *c.backward(ctx, lse))


@pytest.mark.parametrize("s", [70, 300], ids=lambda v: f"s{v}")
@pytest.mark.parametrize("nh,d", STRUCTURES, ids=lambda v: str(v))
def test_padded_rows_may_hold_anything(nh, d, s, mode):
    """Rows at or past n full of NaN and infinities change nothing."""
    c = Case("slopes", mode, 3, nh, s, d, valid=[s // 2 + 3, s - 1, 5])
    ctx, lse = c.forward()
    grads = c.backward(ctx, lse)
    for b, n in enumerate(c.valid):
        c.qkv[:, b, :, n:] = np.where(np.arange(d) % 2, np.nan, np.inf)
        c.dctx[b, n:] = np.nan
    dirty_ctx, dirty_lse = c.forward()
    assert torch.equal(ctx, dirty_ctx) and torch.equal(lse, dirty_lse)
    dirty = c.backward(ctx, lse)
    assert torch.equal(grads[0], dirty[0])


@pytest.mark.parametrize("s", [60, 300], ids=lambda v: f"s{v}")
@pytest.mark.parametrize("low", [-np.inf, float(np.finfo(np.float32).min)])
def test_table_entries_that_hide_keys(low, s, mode):
    """A table entry of -inf, or of the lowest value, gives its keys no weight; rows that it leaves empty are zeros."""
    c = Case("table-one-way-causal", mode, 2, 2, s, 64)
    c.spec.table[:, 0] = low                                  # head 0 sees nothing at all
    c.spec.table[0, 1] = low                                  # head 1 not itself: its first row is empty
    ctx, lse = c.forward()
    c.spec.table[c.spec.table == low] = -np.inf
    got, out = c.shaped(ctx), lse.cpu().numpy()
    with np.errstate(invalid="ignore"):
        ref, ref_lse, _ = SO.forward(c.spec, c.qkv, c.valid)
    assert (got[:, :, 0] == 0).all() and np.isneginf(out[:, 0]).all()
    assert (got[:, 0, 1] == 0).all() and np.isneginf(out[:, 1, 0]).all()
    assert rel_l2(got[:, 1:, 1], ref[:, 1:, 1]) < 2e-3
    assert np.allclose(np.where(np.isfinite(ref_lse), out, 0), np.where(np.isfinite(ref_lse), ref_lse, 0), atol=1e-3)
    dqkv, dtable = c.backward(ctx, lse)
    assert torch.isfinite(dqkv).all() and torch.isfinite(dtable).all()
    assert (dqkv[:, :, 0] == 0).all() and (dtable[:, 0] == 0).all() and dtable[0, 1] == 0


@pytest.mark.parametrize("std", [1e-3, 1.0, 300.0])
def test_gradients_of_any_size(std):
    """FP16 backward with dctx from tiny to large: dU keeps its precision."""
    c = Case("table", "fp16", 2, 2, 150, 64)
    c.dctx = (c.dctx.astype(np.float64) * std).astype(np.float16)
    ctx, lse = c.forward()
    check_backward(c, ctx, lse, *c.backward(ctx, lse))


def test_scores_that_grow_along_the_keys(mode):
    """Row maxima that rise block after block, and then fall."""
    c = Case("plain", mode, 2, 2, 390, 64)
    ramp = np.concatenate([np.linspace(0.1, 4, 200), np.linspace(4, 0.1, 190)])
    c.qkv[1] = (c.qkv[1] * ramp[None, None, :, None]).astype(c.qkv.dtype)
    ctx, lse = c.forward()
    check_forward(c, ctx, lse)
    check_backward(c, ctx, lse, *c.backward(ctx, lse))


def test_results_do_not_change_between_runs(mode):
    c = Case("cap-slopes-table-prefix-docs", mode, 3, 3, 333, 64)
    ctx, lse = c.forward()
    first = c.backward(ctx, lse)
    for _ in range(3):
        again, out = c.forward()
        assert torch.equal(ctx, again) and torch.equal(lse, out)
        assert all(torch.equal(x, y) for x, y in zip(first, c.backward(ctx, lse)))


def test_without_lse_and_on_another_stream(mode):
    c = Case("table", mode, 2, 3, 140, 64)
    ctx, _ = c.forward()
    enc = encoder(3, 64, mode)
    s = torch.cuda.Stream()
    qkv, vl, sc = to_dev(c.qkv), to_dev(c.valid), c.scores()
    out = torch.zeros_like(ctx)
    s.wait_stream(torch.cuda.current_stream())
    enc.op_scored_attention(sc, qkv, vl, out, c.b, c.s, stream=s)
    s.synchronize()
    assert torch.equal(ctx, out)


def test_captured_and_replayed_forward_and_backward(mode):
    """Both calls in a graph of the caller's; the scratch grows between capture and replay."""
    c = Case("table", mode, 2, 4, 130, 32)
    inp = EI.make_inputs(EI.Workload("scored", EI.EncoderShape(4, 32, 64, 1), 1, 1, mode[:4], 1, 1, seed=0))
    enc = encoder_from_inputs(inp)
    enc.set_option("tc_attention", mode != "fp16-simt")
    ctx, lse = c.forward(enc)
    sc, qkv, vl, dctx = c.scores(), to_dev(c.qkv), to_dev(c.valid), to_dev(c.dctx).view(c.b * c.s, -1)
    dqkv, dtable = torch.empty_like(qkv), torch.empty(c.spec.table.shape, device="cuda")
    ctx2, lse2 = torch.empty_like(ctx), torch.empty_like(lse)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())

    def both():
        enc.op_scored_attention(sc, qkv, vl, ctx2, c.b, c.s, lse=lse2)
        enc.op_scored_attention_backward(sc, qkv, vl, ctx2, lse2, dctx, dqkv, c.b, c.s, dtable=dtable)

    with torch.cuda.stream(side):
        g.capture_begin(capture_error_mode="thread_local")
        with pytest.raises(EncError, match="enc_reserve_scored"):
            both()
        g.capture_end()
    torch.cuda.synchronize()
    enc.reserve_scored(c.b, c.s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        g.capture_begin(capture_error_mode="thread_local")
        both()
        g.capture_end()
    torch.cuda.synchronize()
    enc.reserve_scored(8, 4 * c.s)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ctx, ctx2) and torch.equal(lse, lse2)
    want = c.backward(ctx, lse, enc)
    assert torch.equal(want[0], dqkv) and torch.equal(want[1], dtable)
    del g
    enc.close()


# ---------------------------------------------------------------- single-token step
@pytest.mark.parametrize("nh,d", STRUCTURES, ids=lambda v: str(v))
@pytest.mark.parametrize("cap", [1, 2, 63, 200, 1500], ids=lambda v: f"c{v}")
@pytest.mark.parametrize("kind", ["plain", "cap", "slopes", "table-one-way-causal", "docs", "shuffled",
                                  "cap-slopes-table-docs"])
@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
def test_step(dtype, kind, cap, nh, d):
    b = 5
    c = Case(kind, dtype, b, nh, cap, d, seed=cap, valid=[cap] * b)
    r = np.random.default_rng(cap)
    new = r.standard_normal((3, b, nh, 1, d)).astype(c.qkv.dtype)
    length = np.array([0, cap - 1, cap, -1, cap // 2], np.int32)
    cache = np.array(c.qkv[1:])
    for i, n in enumerate(length):                            # what lies past the tokens held is never read
        cache[:, i, :, max(0, min(cap, n)):] = np.nan
    enc = encoder(nh, d, dtype)
    dev, ctx = to_dev(cache), torch.full((b, nh * d), float("nan"), dtype=to_dev(new).dtype, device="cuda")
    enc.op_scored_attention_step(c.scores(), to_dev(new), dev, to_dev(length), ctx, b, cap)
    ref, after = SO.step(c.spec, new, cache, length)
    assert np.array_equal(dev.cpu().numpy(), after, equal_nan=True)
    got = ctx.cpu().numpy().astype(np.float64).reshape(b, nh, d)
    _, eps_out, tiny = _formats(dtype)
    ends = np.where((length >= 0) & (length < cap), length + 1, 0)
    k, v = SO._clean(after[0], ends, 2), SO._clean(after[1], ends, 2)
    dots = c.spec.scale * (np.abs(new[0].astype(np.float64)) @ np.swapaxes(np.abs(k), -1, -2)).max()
    top = dots + np.abs(SO.bias(c.spec, nh, [cap - 1], np.arange(cap))).max() + c.spec.cap
    rel = 2 * ((d + 8) * 2.0 ** -23 * dots + 8 * 2.0 ** -24 * top) + 2.0 ** -20 + (cap + 8) * 2.0 ** -23
    bound = 2 * rel * np.abs(v).max() + eps_out * np.abs(ref) + tiny
    assert (np.abs(got - ref) <= bound).all(), np.max(np.abs(got - ref) / bound)
    assert (got[2] == 0).all() and (got[3] == 0).all()


def test_generation_by_steps_is_the_causal_forward(mode):
    """A run of the calls together: tokens go through the projection and the step one at a time, and give the
    rows that one causal call over all of them gives."""
    nh, d, s, b = 4, 32, 24, 3
    sh = EI.EncoderShape(nh, d, 64, 1)
    inp = EI.make_inputs(EI.Workload("gen", sh, b, s, mode[:4], s, s, seed=3))
    enc = encoder_from_inputs(inp)
    enc.set_option("tc_attention", mode != "fp16-simt")
    c = Case("cap-slopes-table-one-way-causal", mode, b, nh, s, d)
    x, sc = to_dev(inp.x), c.scores()
    qkv = torch.empty((3, b, nh, s, d), dtype=x.dtype, device="cuda")
    enc.op_qkv(0, x, qkv, b, s)
    ctx = torch.empty((b * s, nh * d), dtype=x.dtype, device="cuda")
    enc.op_scored_attention(sc, qkv, to_dev(np.full(b, s, np.int32)), ctx, b, s)
    cache = torch.zeros((2, b, nh, s, d), dtype=x.dtype, device="cuda")
    length = torch.zeros(b, dtype=torch.int32, device="cuda")
    one = torch.empty((3, b, nh, 1, d), dtype=x.dtype, device="cuda")
    for p in range(s):
        enc.op_qkv(0, x[:, p].contiguous(), one, b, 1)
        out = torch.empty((b, nh * d), dtype=x.dtype, device="cuda")
        enc.op_scored_attention_step(sc, one, cache, length, out, b, s)
        length += 1
        ref = ctx.view(b, s, -1)[:, p]
        tol = 1e-2 if mode.startswith("fp16") else 1e-4
        assert rel_l2(out.float().cpu().numpy(), ref.float().cpu().numpy()) < tol
    assert torch.allclose(cache[0].float(), qkv[1].float(), atol=1e-2)
    enc.close()


# ---------------------------------------------------------------- in the encoder forward
def _oracle_stack(inp, spec, nh, d):
    x, vl, layers = inp.as_float64()
    b, s, hid = x.shape
    for lw in layers:
        x2 = x.reshape(b * s, hid)
        qkv = EO.head_split(EO.qkv_projection(x2, lw["w_qkv"], lw["b_qkv"]), b, s, nh, d)
        ctx = SO.forward(spec, qkv, vl)[0].reshape(b * s, hid)
        h1 = EO.bias_residual_layernorm(ctx @ lw["w_o"], lw["b_o"], x2, lw["ln1_g"], lw["ln1_b"])
        u = EO.ffn1_gelu(h1, lw["w_ff1"], lw["b_ff1"])
        x = EO.bias_residual_layernorm(u @ lw["w_ff2"], lw["b_ff2"], h1, lw["ln2_g"], lw["ln2_b"]).reshape(b, s, hid)
    return x


@pytest.mark.parametrize("s", [40, 150], ids=lambda v: f"s{v}")
@pytest.mark.parametrize("kind", ["table", "cap-slopes-table-prefix-docs"])
def test_encoder_forward_with_scores(kind, s, mode):
    nh, d, b = 4, 64, 3
    inp = EI.make_inputs(EI.Workload("stack", EI.EncoderShape(nh, d, 512, 2), b, s, mode[:4], s // 2, s, seed=1))
    enc = encoder_from_inputs(inp)
    enc.set_option("tc_attention", mode != "fp16-simt")
    c = Case(kind, mode, b, nh, s, d)
    x, vl = to_dev(inp.x), to_dev(np.asarray(inp.valid_len, np.int32))
    plain = enc.forward(x, vl)
    sc = c.scores()
    enc.set_scores(sc)
    got = enc.forward(x, vl)
    mask = np.arange(s)[None] < np.asarray(inp.valid_len)[:, None]
    ref = _oracle_stack(inp, c.spec, nh, d)
    tol = 1e-2 if mode.startswith("fp16") else 2e-5
    err = rel_l2(got.cpu().numpy(), ref, mask)
    assert err < tol
    # The scores do something.  With weights of std 0.02 and H = 256, v has std 0.02 sqrt(256) = 0.32, so the
    # attention's share of a layer (a mean of v, times 0.32 again) is a few hundredths of the residual's.
    assert rel_l2(plain.cpu().numpy(), ref, mask) > 5 * err
    # The other entry points run the same thing.
    host = enc.forward_host(inp.x, np.asarray(inp.valid_len, np.int32))
    assert np.array_equal(host[mask], got.cpu().numpy()[mask])
    assert torch.equal(enc.forward_noalloc(x, vl, torch.empty_like(x)), got)
    if c.spec.doc_ids is not None:                            # sized for another batch: refused, not read past its end
        bigger = torch.cat([x, x])
        for call in (lambda: enc.forward(bigger, torch.cat([vl, vl])), lambda: enc.forward(x[:, :-1].contiguous(), vl)):
            with pytest.raises(ValueError, match="shape"):
                call()
    out = torch.empty_like(x)
    rec = enc.record(x, vl, out)
    enc.set_scores(None)
    assert torch.equal(enc.forward(x, vl), plain)
    rec.launch()
    torch.cuda.synchronize()
    assert torch.equal(out, got)
    rec.close()
    if mode.startswith("fp16"):
        enc.set_scores(sc)
        enc.set_packing(True)
        with pytest.raises(EncError, match="ENC_ERR_UNSUPPORTED"):
            enc.forward(x, vl)
        enc.set_packing(False)
        enc.set_option("persistent", True)
        assert torch.equal(enc.forward(x, vl), got)
    enc.close()


# ---------------------------------------------------------------- refusals
def test_refusals():
    enc = handle(4, 32, "fp16")
    c = Case("table", "fp16", 2, 4, 16, 32)
    qkv, vl = to_dev(c.qkv), to_dev(c.valid)
    ctx, lse = torch.empty((32, 128), dtype=torch.float16, device="cuda"), torch.empty((2, 4, 16), device="cuda")
    before = enc.launch_count()

    def bad(match, sc=None, **kw):
        sc = c.scores() if sc is None else sc
        args = dict(qkv=qkv, valid_len=vl, ctx=ctx, batch=2, seq=16, lse=lse)
        args.update(kw)
        with pytest.raises((EncError, ValueError, TypeError), match=match):
            enc.op_scored_attention(sc, **args)

    t = to_dev(c.spec.table)
    bad("num_buckets", Scores(table=t[:1].contiguous(), bidirectional=False))
    bad("num_buckets", Scores(table=t[:7].contiguous()))
    bad("num_buckets", Scores(table=torch.zeros((130, 4), device="cuda")))
    bad("max_distance", Scores(table=t, max_distance=4))
    bad("max_distance", Scores(table=t, max_distance=2049))
    bad("cap", Scores(cap=-1.0))
    bad("cap", Scores(cap=float("nan")))
    bad("cap", Scores(cap=1e-4))
    bad("cap", Scores(cap=2e4))
    bad("scale", Scores(scale=float("inf")))
    bad("causal", Scores(prefix_len=vl))
    bad("overlaps", ctx=qkv[1].view(32, 128))
    bad("shape", Scores(slopes=torch.zeros(3, device="cuda")))
    bad("shape", Scores(doc_ids=torch.zeros((2, 17), dtype=torch.int32, device="cuda")))
    bad("float16", ctx=ctx.float())
    bad("int32", valid_len=vl.long())
    bad("elements", lse=lse[:1].contiguous())
    bad("contiguous", qkv=qkv.transpose(0, 1))
    lib = enc.lib
    sc = c.scores()
    st = torch.cuda.current_stream().cuda_stream
    p = lambda x: x.data_ptr()  # noqa: E731
    assert lib.enc_op_scored_attention(enc.handle, None, p(qkv), p(vl), p(ctx), None, 2, 16, st) == 1
    assert lib.enc_op_scored_attention(enc.handle, sc.pointer, p(qkv) + 2, p(vl), p(ctx), None, 2, 16, st) == 1
    assert lib.enc_op_scored_attention(enc.handle, sc.pointer, p(qkv), p(vl), p(ctx), None, 2, 65537, st) == 2
    assert lib.enc_op_scored_attention(enc.handle, sc.pointer, p(qkv), p(vl), p(ctx), None, 0, 16, st) == 1
    dq = torch.empty_like(qkv)
    plain = Scores()
    assert lib.enc_op_scored_attention_backward(enc.handle, plain.pointer, p(qkv), p(vl), p(ctx), p(lse), p(ctx), p(dq),
                                                p(lse), 2, 16, st) == 1          # dtable without a table
    assert lib.enc_op_scored_attention_backward(enc.handle, plain.pointer, p(qkv), p(vl), p(ctx), None, p(ctx), p(dq),
                                                None, 2, 16, st) == 1
    assert lib.enc_op_scored_attention_backward(enc.handle, plain.pointer, p(qkv), p(vl), p(ctx), p(lse), p(ctx), p(qkv),
                                                None, 2, 16, st) == 1
    assert lib.enc_op_scored_attention_step(enc.handle, plain.pointer, p(qkv), p(qkv), p(vl), p(ctx), 2, 4, st) == 1
    assert enc.launch_count() == before
