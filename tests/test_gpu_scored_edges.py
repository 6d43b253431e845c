"""Attention with modified scores where calls, workspaces and roundings meet: runs of calls without
a wait between them, ragged tiles under a cap, weights and slopes of the smallest sizes, what padded
rows may hold in every form, scratch under memory pressure and capture, overlaps, and tensors that a
caller lets go of.
"""
import numpy as np
import pytest
import torch

import encoder_inputs as EI
from oracle import scored_oracle as SO
from parity_utils import encoder_from_inputs, to_dev
from test_gpu_scored import Case, check_backward, check_forward, encoder
from transformer_encoder_bert_b200 import Scores

pytestmark = pytest.mark.gpu


def fresh_encoder(nh, d, mode):
    """A handle that holds no scratch yet."""
    enc = encoder_from_inputs(EI.make_inputs(EI.Workload("scored", EI.EncoderShape(nh, d, 64, 1), 1, 1, mode[:4], 1, 1, seed=0)))
    enc.set_option("tc_attention", mode != "fp16-simt")
    return enc


# ---------------------------------------------------------------- calls one after the other
@pytest.mark.parametrize("mode", ["fp16", "fp16-simt", "fp32"])
@pytest.mark.parametrize("nh,d,s", [(3, 64, 300), (2, 128, 700), (4, 32, 131)], ids=str)
@pytest.mark.parametrize("pdl", [True, False], ids=["pdl", "no-pdl"])
def test_inputs_that_alternate_through_one_handle(pdl, nh, d, s, mode):
    """Backward calls of different data one behind the other share the scratch: each gets its own statistics."""
    cases = [Case("table-docs", mode, 2, nh, s, d, seed=20 + i, std=(1.0, 0.3, 2.0)[i]) for i in range(3)]
    enc = encoder(nh, d, mode)
    enc.set_option("pdl", pdl)
    try:
        args, want = [], []
        for c in cases:
            ctx, lse = c.forward()
            want.append(c.backward(ctx, lse))
            args.append((c.scores(), to_dev(c.qkv), to_dev(c.valid), ctx, lse, to_dev(c.dctx).view(2 * s, -1)))
        order = [0, 1, 2, 1, 0, 2, 2, 0, 1] * 3
        got = [(torch.empty_like(want[i][0]), torch.empty_like(want[i][1])) for i in order]
        torch.cuda.synchronize()
        for i, (dqkv, dtable) in zip(order, got):
            enc.op_scored_attention_backward(*args[i], dqkv, 2, s, dtable=dtable)
        torch.cuda.synchronize()
    finally:
        enc.set_option("pdl", True)
    assert enc.device_status() == 0
    for i, x in zip(order, got):
        assert torch.equal(want[i][0], x[0]) and torch.equal(want[i][1], x[1])


# ---------------------------------------------------------------- the cap
def equal_scores(mode, s, cap, u, valid, outlier=False):
    """A case whose every score is u (the products are exact), whose v grows along the keys and whose dctx is 1, so
    that all of a far bucket's dT have one sign.  outlier: key 3's score is -2.5 caps instead."""
    d, nh, b = 64, 2, len(valid)
    c = Case("table", mode, b, nh, s, d, seed=30, valid=valid)
    c.spec.cap, c.spec.scale, c.spec.max_distance = float(cap), 0.125, s - 10
    c.spec.table = np.zeros((16, nh), np.float32)
    c.qkv[:2] = 0
    c.qkv[:2, ..., 0] = np.sqrt(u / c.spec.scale)
    c.qkv[2] = (np.arange(1, s + 1) / s)[None, None, :, None]
    if outlier:
        c.qkv[0, ..., 1] = 100
        c.qkv[1, :, :, 3, 1] = -2.5 * cap / c.spec.scale / 100
    c.dctx[:] = 1
    return c


# A score of 0.4 steps (2^-23) of the cap: a tanh that is only good to such a step returns 0 for it, and moves the
# score by 4.8e-4 at a cap of 1e4.  Without that, t, lse (below 8), their forms in log2 and the exponential are off by
# a few 2^-24 of 8, below 2^-19 in all, and sums of s terms by s 2^-24 more.
@pytest.mark.parametrize("mode", ["fp16", "fp16-simt", "fp32"])
@pytest.mark.parametrize("cap", [30.0, 1e4])
@pytest.mark.parametrize("s,valid", [(100, [100, 97, 70]), (150, [150, 129, 141]), (300, [300, 257, 290])], ids=str)
def test_ragged_tiles_keep_small_scores(s, valid, cap, mode):
    """The table's gradient where tiles end in padding: P is rebuilt from the scores that the forward had."""
    c = equal_scores(mode, s, cap, 0.4 * 2.0 ** -23 * cap, valid)
    ctx, lse = c.forward()
    _, dtable = c.backward(ctx, lse)
    _, ref, (p, size, _) = SO.backward(c.spec, c.qkv, c.valid, c.shaped(ctx), lse.cpu().numpy().astype(np.float64), c.dctx)
    rel = 2.0 ** -19 + (s + c.d + 8) * 2.0 ** -24
    bound = np.zeros(ref.shape)
    pos = np.arange(s)
    np.add.at(bound, SO.bucket_matrix(c.spec, pos, pos), np.moveaxis((2 * rel * size).sum(0), 0, -1))
    err = np.abs(dtable.cpu().numpy() - ref)
    assert (err <= bound + 2.0 ** -23 * np.abs(ref)).all(), (err / (bound + 1e-30)).max()


@pytest.mark.parametrize("mode", ["fp16", "fp16-simt", "fp32"])
@pytest.mark.parametrize("cap", [2000.0, 1e4])
@pytest.mark.parametrize("s,valid", [(100, [100, 97, 70]), (128, [128, 64, 128]), (300, [300, 257, 290])], ids=str)
def test_small_scores_beside_a_large_one(s, valid, cap, mode):
    """One key far past the cap does not change how the others' scores are formed."""
    c = equal_scores(mode, s, cap, 0.4 * 2.0 ** -23 * cap, valid, outlier=True)
    ctx, lse = c.forward()
    ref, ref_lse, _ = SO.forward(c.spec, c.qkv, c.valid)
    got = lse.cpu().numpy().astype(np.float64)
    seen = np.isfinite(ref_lse)
    # lse is near log n: the sum is off by n 2^-24, and t, its maximum and the logarithm by a few 2^-24 of 8.
    assert np.abs(got[seen] - ref_lse[seen]).max() <= (s + 64) * 2.0 ** -24
    # The same for the gradient's P: dv sums n of them, each rounded once in FP16 mode, and is rounded once.
    dqkv, _ = c.backward(ctx, lse)
    want = SO.backward(c.spec, c.qkv, c.valid, c.shaped(ctx), got, c.dctx)[0]
    rel = (s + 64) * 2.0 ** -23 + (2.0 ** -10 if mode.startswith("fp16") else 2.0 ** -23)
    assert (np.abs(dqkv[2].cpu().numpy() - want[2]) <= rel * np.abs(want[2]) + 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
@pytest.mark.parametrize("cap", [30.0, 1e3, 1e4])
@pytest.mark.parametrize("capacity", [100, 600])
def test_step_keeps_small_scores(capacity, cap, dtype):
    """Half of the keys score u, half -u, with values 1 and -1: ctx = tanh(u), which a tanh good to a step (2^-23) of
    the cap rounds to nothing."""
    nh, d, b = 2, 64, 2
    enc = encoder(nh, d, dtype)
    np_dt = np.float16 if dtype == "fp16" else np.float32
    a = np_dt(np.sqrt(0.45 * 2.0 ** -23 * cap / 0.125))
    new, cache = np.zeros((3, b, nh, 1, d), np_dt), np.zeros((2, b, nh, capacity, d), np_dt)
    sign = np.where(np.arange(capacity) % 2, -1.0, 1.0)
    new[0, ..., 0] = a
    cache[0, ..., 0] = (sign * a)[None, None]
    cache[1] = sign[None, None, :, None]
    length = np.array([capacity - 1, 59], np.int32)           # the new token, of the odd positions, is the last -u
    new[1, ..., 0], new[2] = -a, -1
    ctx = torch.empty((b, nh * d), dtype=to_dev(new).dtype, device="cuda")
    enc.op_scored_attention_step(Scores(scale=0.125, cap=cap), to_dev(new), to_dev(cache), to_dev(length), ctx, b, capacity)
    u = cap * np.tanh(float(a) * float(a) * 0.125 / cap)
    # A weight is 1 -+ 2u with an error of 2^-22 (its exponential), the two sums' of (capacity / 4) 2^-24 or less; then
    # 2^-20 of u and the rounding of the result.
    tol = 2.0 ** -21 + capacity * 2.0 ** -24 / 4 + (2.0 ** -20 + (2.0 ** -11 if dtype == "fp16" else 2.0 ** -23)) * u + 2.0 ** -25
    assert np.abs(ctx.cpu().numpy().astype(np.float64) - np.tanh(u)).max() <= tol


@pytest.mark.parametrize("mode", ["fp16", "fp16-simt", "fp32"])
@pytest.mark.parametrize("cap", [1.0, 100.0])
@pytest.mark.parametrize("s", [90, 300])
def test_gradients_through_saturated_scores(s, cap, mode):
    """Every score 5 to 8 caps out, where 1 - tanh^2 is 2e-4 to 5e-7 and tanh itself has no digits left for it."""
    nh, d, b = 2, 64, 2
    c = Case("plain", mode, b, nh, s, d, seed=31, valid=[s, s - 7])
    c.spec.scale, c.spec.cap = 0.125, cap
    r = np.random.default_rng(32)
    c.qkv[:2] = 0
    c.qkv[0, ..., 0] = r.uniform(7, 8, (b, nh, s))            # scale q k = q k / 8 in +-[5, 8] caps
    c.qkv[1, ..., 0] = r.uniform(5.75, 8, (b, nh, s)) * r.choice([-1.0, 1.0], (b, nh, s)) * cap
    if cap == 100.0:                                          # (the keys below the cap would get no weight)
        c.qkv[1] = np.abs(c.qkv[1])
    c.dctx = (c.dctx * 30).astype(c.dctx.dtype)
    ctx, lse = c.forward()
    dqkv, _ = c.backward(ctx, lse)
    ref, _, (p, size, du) = SO.backward(c.spec, c.qkv, c.valid, c.shaped(ctx), lse.cpu().numpy().astype(np.float64), c.dctx)
    q, k = (np.abs(SO._clean(c.qkv[i], c.valid, 2)) for i in range(2))
    x = 0.125 * (q @ np.swapaxes(k, -1, -2)) / cap
    slope = np.where(p > 0, 1 / np.cosh(np.minimum(x, 300)) ** 2, 0)
    # x is off by 3 roundings and 2^-24 of its exponent's rounding: 2^-21 of 8, twice that for the slope, whose own
    # operations add 2^-20; P by t (4 roundings of 1.5 cap, tanh 2^-22 of the cap) and 2^-19; sums of s terms by s 2^-24.
    rel = 2.0 ** -17 + cap * 2.0 ** -20 + 2.0 ** -19 + (s + d) * 2.0 ** -24
    half = 2.0 ** -11 if mode.startswith("fp16") else 0.0
    # FP16: dU is scaled so that the largest |dctx_i| |v_j| is at 2^13 or more, and below 2^-14 its halves are off by 2^-25.
    do, v = (SO._clean(a, c.valid, i) for a, i in ((c.dctx, 1), (c.qkv[2], 2)))
    norm = np.sqrt((do ** 2).sum(-1)).max() * np.sqrt((v ** 2).sum(-1)).max()
    step = (2.0 ** -25 * 2.0 ** -13 * 2 * norm if mode == "fp16" else 0.0) * (p > 0)
    err = half * np.abs(du) + 2 * rel * size * slope + step
    out = 2.0 ** -11 if half else 2.0 ** -24
    for i, want in ((0, 0.125 * (err @ k)), (1, 0.125 * (np.swapaxes(err, -1, -2) @ q))):
        bound = want + out * np.abs(ref[i]) + (2.0 ** -25 if half else 0.0)
        got = np.abs(dqkv[i].cpu().numpy() - ref[i])
        assert (got <= bound + 1e-30).all(), (i, (got / (bound + 1e-30)).max())


# ---------------------------------------------------------------- scratch
def test_scratch_grows_by_what_is_needed_when_memory_is_short():
    """Scratch grows by doubling, but a device without room for twice the old size still serves a little more than it."""
    enc = fresh_encoder(4, 32, "fp32")
    filler = None
    try:
        torch.cuda.empty_cache()                              # (what other tests left in PyTorch's cache)
        free = torch.cuda.mem_get_info()[0]
        enc.reserve_scored(4096, 4096)
        held = free - torch.cuda.mem_get_info()[0]            # 0.8 GB
        assert held > 2 ** 29
        filler = torch.empty(torch.cuda.mem_get_info()[0] - held - held // 2, dtype=torch.uint8, device="cuda")
        enc.reserve_scored(4300, 4096)
    finally:
        filler = None
        enc.close()
        torch.cuda.empty_cache()


def held_outside_torch():
    """Device bytes in use that PyTorch's allocator does not hold: the library's, and the context's."""
    torch.cuda.synchronize()
    free, total = torch.cuda.mem_get_info()
    return total - free - torch.cuda.memory_reserved()


def test_calls_without_scratch_allocate_nothing():
    """The backward of up to 128 positions without dtable uses no scratch: it runs under capture on a fresh handle."""
    c = Case("table", "fp16", 2, 4, 100, 32, seed=33)
    ctx, lse = c.forward()
    want = c.backward(ctx, lse)[0]
    enc = fresh_encoder(4, 32, "fp16")
    sc, qkv, vl, dctx = c.scores(), to_dev(c.qkv), to_dev(c.valid), to_dev(c.dctx).view(200, -1)
    dqkv = torch.empty_like(qkv)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g.capture_begin(capture_error_mode="thread_local")
        try:
            enc.op_scored_attention_backward(sc, qkv, vl, ctx, lse, dctx, dqkv, 2, 100)
        finally:
            g.capture_end()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(dqkv, want)
    held = held_outside_torch()
    enc.op_scored_attention_backward(sc, qkv, vl, ctx, lse, dctx, dqkv, 2, 100)
    assert held_outside_torch() == held
    del g
    enc.close()


@pytest.mark.parametrize("mode", ["fp16", "fp16-simt", "fp32"])
@pytest.mark.parametrize("s", [100, 300])
def test_reserved_scratch_serves_every_call_of_its_shape(s, mode):
    """After a reservation neither the largest table's gradient nor another kernel choice has to allocate."""
    enc = fresh_encoder(3, 64, mode)
    enc.reserve_scored(2, s)
    for m in ([mode] if mode == "fp32" else ["fp16", "fp16-simt"]):
        c = Case("table", m, 2, 3, s, 64, seed=34)
        c.spec.table = np.random.default_rng(1).standard_normal((128, 3)).astype(np.float32)
        c.spec.max_distance = 90
        ctx, lse = c.forward()
        want = c.backward(ctx, lse)
        held = held_outside_torch()
        enc.set_option("tc_attention", m != "fp16-simt")
        got = c.backward(ctx, lse, enc)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
        assert held_outside_torch() == held
    enc.close()


# ---------------------------------------------------------------- buffers that overlap
@pytest.mark.parametrize("mode", ["fp16", "fp32"])
def test_overlaps_are_refused(mode):
    """Whatever a call writes may not lie over what it reads, or over what else it writes."""
    b, nh, s, d = 2, 4, 16, 32
    enc = encoder(nh, d, mode)
    lib, st = enc.lib, torch.cuda.current_stream().cuda_stream
    size = 2 if mode == "fp16" else 4
    act, stat = b * s * nh * d * size, b * s * nh * 4
    names = dict(qkv=3 * act, ctx=act, dctx=act, dqkv=3 * act, lse=stat, valid=4 * b, slopes=4 * nh, table=16 * nh * 4,
                 dtable=16 * nh * 4, prefix=4 * b, docs=4 * b * s, cache=2 * act // s * 3, new=3 * act // s)
    step = dict(names, ctx=act // s, docs=4 * b * 3)
    block = torch.zeros(sum(-(-n // 256) * 256 for n in names.values()), dtype=torch.uint8, device="cuda")
    at, place = block.data_ptr(), {}
    for name, n in names.items():
        place[name] = at
        at += -(-n // 256) * 256

    def call(op, **moved):
        p = dict(place, **moved)
        sc = Scores(causal=True)
        c = sc.c
        c.slopes, c.bias_table, c.num_buckets, c.max_distance = p["slopes"], p["table"], 16, 128
        c.prefix_len, c.doc_ids = p["prefix"], p["docs"]
        if op == "forward":
            return lib.enc_op_scored_attention(enc.handle, sc.pointer, p["qkv"], p["valid"], p["ctx"], p["lse"], b, s, st)
        if op == "backward":
            return lib.enc_op_scored_attention_backward(enc.handle, sc.pointer, p["qkv"], p["valid"], p["ctx"], p["lse"],
                                                        p["dctx"], p["dqkv"], p["dtable"], b, s, st)
        return lib.enc_op_scored_attention_step(enc.handle, sc.pointer, p["new"], p["cache"], p["valid"], p["ctx"], b, 3, st)

    scores = ["slopes", "table", "prefix", "docs"]
    uses = dict(forward=(["ctx", "lse"], ["qkv", "valid"] + scores),
                backward=(["dqkv", "dtable"], ["qkv", "ctx", "dctx", "lse", "valid"] + scores),
                step=(["cache", "ctx"], ["new", "valid"] + scores))
    before = enc.launch_count()
    for op, (written, read) in uses.items():
        sizes = step if op == "step" else names
        for i, w in enumerate(written):
            for o in read + written[:i]:
                start = place[o] + (sizes[o] - 1) // 16 * 16  # over the last bytes of o
                assert call(op, **{w: start}) == 1, (op, w, o)
                assert "overlaps" in lib.enc_last_error().decode()
                if w in ("ctx", "lse", "dtable"):             # and o over the last bytes of w
                    start = place[w] + (sizes[w] - 1) // 16 * 16
                    assert call(op, **{o: start}) == 1, (op, o, w)
    assert enc.launch_count() == before
    for op in uses:
        assert call(op) == 0
    torch.cuda.synchronize()
    assert enc.device_status() == 0


# ---------------------------------------------------------------- tensors that a caller lets go of
@pytest.mark.parametrize("how", ["forward", "host_async"])
@pytest.mark.parametrize("as_handle", [False, True], ids=["stream", "handle"])
def test_scores_outlive_forwards_in_flight(as_handle, how):
    """Replacing the scores while a forward on another stream still waits does not give their memory to the next tensor."""
    nh, d, b, s = 4, 32, 2, 40
    inp = EI.make_inputs(EI.Workload("stack", EI.EncoderShape(nh, d, 64, 2), b, s, "fp16", s, s, seed=1))
    enc = encoder_from_inputs(inp)
    x, vl = to_dev(inp.x), to_dev(np.asarray(inp.valid_len, np.int32))
    want = enc.forward(x, vl)
    out, side = torch.empty_like(x), torch.cuda.Stream()
    host = [t.cpu().pin_memory() for t in (x, vl, out)]
    table = torch.zeros((32, nh), device="cuda")              # (zeros: the scores stay the plain ones)
    docs = torch.zeros((b, s), dtype=torch.int32, device="cuda")
    places = {table.data_ptr(), docs.data_ptr()}
    sc = Scores(table=table, doc_ids=docs)
    enc.set_scores(sc)
    enc.forward(x, vl)                                        # (everything is loaded and allocated)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)                        # about 0.2 s
    st = side.cuda_stream if as_handle else side
    if how == "forward":
        enc.forward(x, vl, out=out, stream=st)
    else:
        enc.forward_host_async_ptr(*(t.data_ptr() for t in host), b, s, stream=st)
        enc.host_join(st)
    enc.set_scores(None)
    busy = not side.query()
    del sc, table, docs
    fresh = [torch.empty((32, nh), device="cuda") for _ in range(8)] + [torch.empty((b, s), device="cuda") for _ in range(8)]
    assert busy and not side.query()
    assert places.isdisjoint(t.data_ptr() for t in fresh)
    torch.cuda.synchronize()
    got = (host[2] if how == "host_async" else out).float().cpu().numpy()
    assert np.abs(got - want.float().cpu().numpy()).max() < 0.05
    assert enc.device_status() == 0
    enc.close()


# ---------------------------------------------------------------- small weights
def seldom_attended(mode, d, s, bits, v=1.0, do=1.0):
    """Key 0 takes nearly all of every row, the others about 2^-bits each."""
    b, nh = 2, 2
    c = Case("plain", mode, b, nh, s, d, seed=35, valid=[s, s - 9])
    c.spec.scale = 1.0
    c.qkv[:2] *= 0.01
    c.qkv[:2, ..., 0] = 0
    c.qkv[0, ..., 0] = 1
    c.qkv[1, :, :, 0, 0] = bits * np.log(2)
    c.qkv[2] = (np.abs(c.qkv[2]) + 1).astype(c.qkv.dtype) * c.qkv.dtype.type(v)
    c.qkv[2, :, :, 0] = 0
    c.dctx = (np.abs(c.dctx) + 1).astype(c.dctx.dtype) * c.dctx.dtype.type(do)
    return c


@pytest.mark.parametrize("mode", ["fp16", "fp16-simt", "fp32"])
@pytest.mark.parametrize("bits", [16, 22, 26])
@pytest.mark.parametrize("d,s", [(64, 100), (64, 300), (32, 300), (128, 128), (128, 300)], ids=str)
def test_gradient_of_seldom_attended_keys(d, s, bits, mode):
    """dv of keys whose weights are far below FP16's smallest numbers."""
    c = seldom_attended(mode, d, s, bits, do=500.0)
    ctx, lse = c.forward()
    dqkv, _ = c.backward(ctx, lse)
    ref, _, (p, _, _) = SO.backward(c.spec, c.qkv, c.valid, c.shaped(ctx), lse.cpu().numpy().astype(np.float64), c.dctx)
    # t is below 20 and off by (d + 8) 2^-23 of that or less, 2^-21 more for its log2 form and the exponential; a weight
    # is rounded once (2^-11) in FP16 mode, as 2^13 of itself, which is 2^-13 or more here; all terms have one sign.
    half = mode.startswith("fp16")
    rel = 20 * (d + 8) * 2.0 ** -23 + 20 * 2.0 ** -22 + s * 2.0 ** -23 + (2.0 ** -10 if half else 2.0 ** -23)
    got, want = dqkv[2, :, :, 1:].cpu().numpy(), ref[2][:, :, 1:]       # (key 0's own sum may pass 65504)
    err = np.abs(got - want)
    assert (err <= rel * np.abs(want) + (2.0 ** -25 if half else 0)).all(), (err / (np.abs(want) + 1e-30)).max()


@pytest.mark.parametrize("mode", ["fp16", "fp32"])
@pytest.mark.parametrize("d,s,bits", [(64, 128, 20), (64, 16384, 25.7), (128, 16384, 25.7), (32, 9000, 25.7)], ids=str)
def test_many_small_weights_add_up(d, s, bits, mode):
    """Weights that FP16 would round to nothing beside the row's largest, which has a v of 0."""
    b, nh = 1, 2
    enc = encoder(nh, d, mode)
    dt = torch.float16 if mode == "fp16" else torch.float32
    qkv = torch.zeros((3, b, nh, s, d), dtype=dt, device="cuda")
    qkv[0, ..., 0] = 1
    qkv[1, :, :, 0, 0] = bits * np.log(2)
    qkv[2] = torch.linspace(1, 2, d, device="cuda").to(dt)
    qkv[2, :, :, 0] = 0
    ctx, lse = torch.empty((b * s, nh * d), dtype=dt, device="cuda"), torch.empty((b, nh, s), device="cuda")
    enc.op_scored_attention(Scores(scale=1.0), qkv, torch.tensor([s], dtype=torch.int32, device="cuda"), ctx, b, s, lse=lse)
    assert enc.device_status() == 0
    w = np.exp(-float(qkv[1, 0, 0, 0, 0]))
    v = qkv[2, 0, 0, 1].double().cpu().numpy()
    ref = (s - 1) * w / (1 + (s - 1) * w) * v
    got = ctx.double().cpu().numpy().reshape(s, nh, d)
    # FP16: a weight of 2^-25.7 is 2^-18.7 as it is rounded, to a multiple of 2^-24: off by 2^-25, a 75th of it (of 2^-20,
    # 2^-5, by 2^-11); and the result is rounded once (2^-25 below 2^-14).  t: one product of a value below 18, 2^-22
    # for its log2 form and 2^-22 for the exponential; sums of s equal terms: s 2^-24.
    if mode == "fp16":
        rel = (2.0 ** -25 / 2.0 ** -18.8 if bits > 25 else 2.0 ** -11) + 2.0 ** -11 + 2.0 ** -17 + s * 2.0 ** -24
        tol = rel * ref + 2.0 ** -25
    else:
        tol = (2.0 ** -17 + s * 2.0 ** -24) * ref
    assert (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) / tol).max()
    want = float(qkv[1, 0, 0, 0, 0]) + np.log1p((s - 1) * w)
    assert np.abs(lse.double().cpu().numpy() - want).max() <= 2.0 ** -20 * 18 + s * 2.0 ** -24


# ---------------------------------------------------------------- padded rows
@pytest.mark.parametrize("mode", ["fp16", "fp16-simt", "fp32"])
@pytest.mark.parametrize("kind", ["cap", "table", "docs", "cap-table-shuffled", "cap-slopes-table-prefix-docs"])
@pytest.mark.parametrize("nh,d,s,valid", [(3, 64, 70, [37, 69, 5, 16]), (2, 128, 128, [127, 65, 33, 1]), (4, 32, 100, [90, 40, 64, 0]),
                                          (3, 64, 300, [153, 299, 5, 257]), (2, 128, 300, [130, 201, 64, 290]),
                                          (4, 32, 200, [199, 129, 17, 0])], ids=str)
def test_padded_rows_may_hold_anything_in_every_form(nh, d, s, valid, kind, mode):
    """NaN and infinities in rows at or past n, and any document ids there, change no bit of any output."""
    c = Case(kind, mode, len(valid), nh, s, d, seed=36, valid=valid)
    ctx, lse = c.forward()
    grads = c.backward(ctx, lse)
    r = np.random.default_rng(37)
    for b, n in enumerate(valid):
        c.qkv[:, b, :, n:] = np.where(np.arange(d) % 2, np.nan, np.where(np.arange(d) % 4, np.inf, -np.inf))
        c.dctx[b, n:] = np.where(np.arange(d) % 2, np.inf, np.nan)
        if c.spec.doc_ids is not None:
            c.spec.doc_ids[b, n:] = r.integers(-(2 ** 31), 2 ** 31, s - n)
    dirty_ctx, dirty_lse = c.forward()
    assert torch.equal(ctx, dirty_ctx) and torch.equal(lse, dirty_lse)
    dirty = c.backward(ctx, lse)
    assert torch.equal(grads[0], dirty[0])
    if grads[1] is not None:
        assert torch.isfinite(dirty[1]).all() and torch.equal(grads[1], dirty[1])


@pytest.mark.parametrize("mode", ["fp16", "fp16-simt", "fp32"])
@pytest.mark.parametrize("sign", [1, -1], ids=["rising", "falling"])
@pytest.mark.parametrize("size", [5e7, 1.4e8, 1e9], ids=str)
@pytest.mark.parametrize("d,s", [(64, 100), (64, 300), (32, 300), (128, 128), (128, 700)], ids=str)
def test_scores_of_any_finite_size(d, s, size, sign, mode):
    """Scores up to 10^9, further apart than their rounding: each row is its largest key's.  (Where floats are 8 or 16
    apart, a 7 or 15 added to one becomes a factor of 2 or 256.)"""
    c = Case("plain", mode, 2, 2, s, d, seed=38, valid=[s, s - 3])
    c.spec.scale = float(np.float32(size / (16384 * 16 * (s // 2))))
    c.qkv[:2] = 0
    c.qkv[0, ..., 0] = 16384
    c.qkv[1, ..., 0] = (sign * 16 * np.arange(-(s // 2), s - s // 2))[None, None]
    ctx, lse = c.forward()
    got, out = c.shaped(ctx), lse.cpu().numpy()
    for b, n in enumerate(c.valid):
        best = n - 1 if sign > 0 else 0
        want = np.broadcast_to(c.qkv[2, b, :, best].astype(np.float64), (n, 2, d))
        assert np.array_equal(got[b, :n], want)
        top = c.spec.scale * 16384 * float(c.qkv[1, b, 0, best, 0])
        assert (np.abs(out[b, :, :n] - top) <= 2.0 ** -22 * abs(top) + 1e-6).all()


@pytest.mark.parametrize("cap,std", [(100.0, 6.0), (1e4, 40.0)])
@pytest.mark.parametrize("kind", ["cap", "cap-slopes", "cap-docs", "cap-table-one-way-causal", "cap-slopes-table-prefix-docs"])
@pytest.mark.parametrize("nh,d,s", [(3, 64, 90), (3, 64, 300), (2, 128, 128), (2, 128, 260), (4, 32, 70), (4, 32, 200)], ids=str)
def test_large_caps_in_every_form(nh, d, s, kind, cap, std):
    """The kernels of caps above 64: scores from near nothing to past the cap."""
    c = Case(kind, "fp16", 2, nh, s, d, seed=39, std=std)
    c.spec.cap = cap
    c.qkv[2] = (c.qkv[2] / std).astype(np.float16)
    ctx, lse = c.forward()
    check_forward(c, ctx, lse)
    check_backward(c, ctx, lse, *c.backward(ctx, lse))
