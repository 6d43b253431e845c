"""Pins of the scored-attention oracle (CPU), and what the binding refuses without a GPU."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

from oracle import encoder_oracle as EO
from oracle import scored_oracle as SO
from transformer_encoder_bert_b200 import binding as B


def _rand(shape, seed):
    return np.random.default_rng(seed).standard_normal(shape)


def _spec(kind, b, s, nh, d=8):
    r = np.random.default_rng(5)
    spec = SO.ScoreSpec(scale=0.3)
    if "cap" in kind:
        spec.cap = 1.5
    if "slopes" in kind:
        spec.slopes = r.uniform(0.05, 0.5, nh)
    if "table" in kind:
        spec.table, spec.max_distance = r.standard_normal((8, nh)), 9
    if "causal" in kind:
        spec.causal = True
    if "prefix" in kind:
        spec.causal, spec.prefix_len = True, r.integers(0, s, b)
    if "docs" in kind:
        spec.doc_ids = np.sort(r.integers(0, 3, (b, s)), 1)
    return spec


KINDS = ["plain", "cap", "slopes", "table", "causal", "prefix", "docs", "cap-slopes-table-prefix-docs"]


def test_without_modifications_it_is_the_encoders_attention():
    qkv = _rand((3, 2, 3, 7, 8), 1)
    spec = SO.ScoreSpec(scale=8 ** -0.5)
    vl = np.array([7, 4])
    ctx, lse, _ = SO.forward(spec, qkv, vl)
    ref = EO.attention(qkv, vl).reshape(2, 7, 3, 8)
    assert np.allclose(ctx[0], ref[0], atol=1e-12) and np.allclose(ctx[1, :4], ref[1, :4], atol=1e-12)
    assert (ctx[1, 4:] == 0).all() and np.isneginf(lse[1, :, 4:]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_forward_against_scalar_loops(kind):
    b, nh, s, d = 2, 2, 9, 8
    qkv, spec, vl = _rand((3, b, nh, s, d), 2), _spec(kind, 2, 9, 2), np.array([9, 6])
    ctx, lse, _ = SO.forward(spec, qkv, vl)
    for bb, h, i in itertools.product(range(b), range(nh), range(s)):
        ws, vs = [], []
        for j in range(s):
            if i >= vl[bb] or j >= vl[bb]:
                continue
            if spec.causal and j > i and not (spec.prefix_len is not None and j < spec.prefix_len[bb]):
                continue
            if spec.doc_ids is not None and spec.doc_ids[bb, i] != spec.doc_ids[bb, j]:
                continue
            u = spec.scale * float(qkv[0, bb, h, i] @ qkv[1, bb, h, j])
            if spec.cap:
                u = spec.cap * np.tanh(u / spec.cap)
            if spec.slopes is not None:
                u -= spec.slopes[h] * abs(j - i)
            if spec.table is not None:
                u += spec.table[SO.bucket(j - i, 8, 9, True), h]
            ws.append(np.exp(u))
            vs.append(qkv[2, bb, h, j])
        if not ws:
            assert (ctx[bb, i, h] == 0).all() and lse[bb, h, i] == -np.inf
        else:
            assert np.allclose(ctx[bb, i, h], np.tensordot(ws, vs, 1) / sum(ws), atol=1e-12)
            assert np.isclose(lse[bb, h, i], np.log(sum(ws)), atol=1e-12)


@pytest.mark.parametrize("kind", KINDS)
def test_backward_against_differences_and_autograd(kind):
    b, nh, s, d = 2, 2, 6, 4
    spec, vl = _spec(kind, b, s, nh), np.array([6, 4])
    qkv, dctx = _rand((3, b, nh, s, d), 3), _rand((b, s, nh, d), 4)
    ctx, lse, _ = SO.forward(spec, qkv, vl)
    dqkv, dtable, _ = SO.backward(spec, qkv, vl, ctx, lse, dctx)
    loss = lambda x: float((SO.forward(spec, x, vl)[0] * SO._clean(dctx, vl, 1)).sum())  # noqa: E731
    eps = 1e-5
    for idx in [(0, 0, 0, 0, 0), (0, 1, 1, 3, 2), (1, 0, 1, 2, 3), (1, 1, 0, 0, 1), (2, 0, 0, 5, 0), (2, 1, 1, 5, 0)]:
        up, dn = qkv.copy(), qkv.copy()
        up[idx] += eps
        dn[idx] -= eps
        assert abs((loss(up) - loss(dn)) / (2 * eps) - dqkv[idx]) < 1e-8
    if spec.table is not None:
        for idx in [(0, 0), (1, 1), (5, 0), (3, 1)]:
            at = spec.table[idx]
            spec.table[idx] = at + eps
            up = loss(qkv)
            spec.table[idx] = at - eps
            dn = loss(qkv)
            spec.table[idx] = at
            assert abs((up - dn) / (2 * eps) - dtable[idx]) < 1e-8
    x = torch.tensor(qkv, requires_grad=True)                 # autograd over the dense formula
    u = spec.scale * x[0] @ x[1].transpose(-1, -2)
    if spec.cap:
        u = spec.cap * torch.tanh(u / spec.cap)
    t = u + torch.tensor(SO.bias(spec, nh, np.arange(s), np.arange(s)))
    see = torch.tensor(SO.visible(spec, vl, b, s))[:, None]
    p = torch.softmax(t.masked_fill(~see, -1e300), -1) * see
    (p @ x[2]).transpose(1, 2).backward(torch.tensor(SO._clean(dctx, vl, 1)))
    assert np.allclose(x.grad.numpy(), dqkv, atol=1e-12)


@pytest.mark.parametrize("kind", ["plain", "cap", "slopes", "table", "docs"])
def test_steps_are_the_rows_of_a_causal_forward(kind):
    b, nh, s, d = 2, 2, 7, 8
    spec = _spec(kind + "-causal", b, s, nh)
    qkv = _rand((3, b, nh, s, d), 6)
    ctx, _, _ = SO.forward(spec, qkv, [s, s])
    cache = np.full((2, b, nh, s, d), np.nan)
    for p in range(s):
        out, cache = SO.step(spec, qkv[:, :, :, p:p + 1], cache, [p, p])
        assert np.allclose(out, ctx[:, p], atol=1e-12)
    out, after = SO.step(spec, qkv[:, :, :, :1], cache, [-1, s])
    assert (out == 0).all() and (after == cache).all()


def test_bucket_borders():
    """Exact powers fall into the upper bucket; the last bucket starts no later than max_distance."""
    assert [SO.bucket(-a, 32, 128, True) for a in (0, 7, 8, 11, 12, 15, 16, 22, 23, 31, 32, 45, 46, 63, 64, 90, 91, 127, 128, 9999)] == \
        [0, 7, 8, 8, 9, 9, 10, 10, 11, 11, 12, 12, 13, 13, 14, 14, 15, 15, 15, 15]
    assert SO.bucket(3, 32, 128, True) == 19 and SO.bucket(3, 32, 128, False) == 0
    assert SO.bucket(-200, 32, 128, False) == 31
    for nb, md, both in [(2, 5, False), (4, 2, True), (16, 64, True), (64, 2048, True), (128, 100, False)]:
        seen = [SO.bucket(-a, nb, md, both) for a in range(md + 3)]
        m = nb // 2 if both else nb
        assert seen[0] == 0 and seen[md] == m - 1 and all(0 <= y - x for x, y in zip(seen, seen[1:]))


def test_entry_points_refuse_a_null_handle():
    lib = B.load_library()
    assert lib.enc_set_scores(None, None) == 1
    assert lib.enc_reserve_scored(None, 1, 1) == 1
    assert lib.enc_op_scored_attention(None, None, None, None, None, None, 1, 1, None) == 1
    assert lib.enc_op_scored_attention_backward(None, None, None, None, None, None, None, None, None, 1, 1, None) == 1
    assert lib.enc_op_scored_attention_step(None, None, None, None, None, None, 1, 1, None) == 1
    assert b"null handle" in lib.enc_last_error()


def test_scores_struct_matches_the_header_and_refuses_host_tensors():
    import os
    import re
    text = open(os.path.join(os.path.dirname(B.__file__), "..", "include", "enc.h")).read()
    body = text[text.rindex("typedef struct {"):text.index("} enc_scores;")]
    fields = re.findall(r"(?:float|int|const float\*|const int32_t\*)\s+(\w+);", body)
    assert tuple(fields) == tuple(name for name, _ in B.EncScores._fields_)
    assert ctypes.sizeof(B.EncScores) == 56
    with pytest.raises(TypeError):
        B.Scores(slopes=torch.zeros(4))
    with pytest.raises(TypeError):
        B.Scores(doc_ids=np.zeros((1, 4), np.int32))


class _FakeTensor:
    """What the binding looks at, of a CUDA tensor on another device."""

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self._device = shape, dtype, device
        self.is_cuda = True

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(np.prod(self.shape))

    def get_device(self):
        return self._device


def test_tensors_of_another_device_or_shape_are_refused():
    ok = _FakeTensor((2, 4), torch.float32, 0)
    assert B._shaped_ptr(ok, "float32", 8, 0) == 1 << 20
    with pytest.raises(ValueError, match="cuda:1"):
        B._shaped_ptr(_FakeTensor((2, 4), torch.float32, 1), "float32", 8, 0)
    with pytest.raises(ValueError, match="float16"):
        B._shaped_ptr(ok, "float16", 8, 0)
    with pytest.raises(ValueError, match="elements"):
        B._shaped_ptr(ok, "float32", 9, 0)
    sc = B.Scores(table=_FakeTensor((8, 4), torch.float32, 1), causal=True,
                  prefix_len=_FakeTensor((3,), torch.int32, 1), doc_ids=_FakeTensor((3, 5), torch.int32, 1))
    sc.check(4, 1, 3, 5)
    for args, match in (((4, 0, 3, 5), "device"), ((5, 1, 3, 5), "table"), ((4, 1, 2, 5), "prefix_len"),
                        ((4, 1, 3, 6), "doc_ids")):
        with pytest.raises(ValueError, match=match):
            sc.check(*args)
    with pytest.raises(ValueError, match="int32"):
        B.Scores(doc_ids=_FakeTensor((3, 5), torch.int64, 0))
