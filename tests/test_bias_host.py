"""Host-side checks of the relative bias: refusals before any CUDA call,
workspace sizes, and the bucket maker against its definition."""
import ctypes

import pytest
import torch

from head_context_attention_gb300 import inputs, ops

W = inputs.WORKLOADS["tiny-gqa-s1k"]
PTR = 1 << 20    # never dereferenced: every call below fails before any CUDA call


def _desc(**kw):
    d = ops.make_desc(W)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("buckets,status", [
    (ops.RelBuckets(4, [1, 2, 3]), ops.LOONG_OK),
    (ops.RelBuckets(1, []), ops.LOONG_OK),
    (ops.RelBuckets(2, [-5, 5], [1, 0, 1]), ops.LOONG_OK),
    (ops.RelBuckets(3, [1, 2, 3]), ops.LOONG_ERR_INVALID_ARG),          # interval 3 has no bucket
    (ops.RelBuckets(4, [1, 3, 2]), ops.LOONG_ERR_INVALID_ARG),          # not increasing
    (ops.RelBuckets(4, [1, 1, 2]), ops.LOONG_ERR_INVALID_ARG),
    (ops.RelBuckets(0, []), ops.LOONG_ERR_INVALID_ARG),
    (ops.RelBuckets(257, []), ops.LOONG_ERR_INVALID_ARG),
    (ops.RelBuckets(256, list(range(1, 256))), ops.LOONG_OK),
    (ops.RelBuckets(256, list(range(1, 257)), [0] * 257), ops.LOONG_ERR_INVALID_ARG),   # 257 intervals
    (ops.RelBuckets(2, [1], [0, 2]), ops.LOONG_ERR_INVALID_ARG),
    (ops.RelBuckets(2, [1], [0, -1]), ops.LOONG_ERR_INVALID_ARG),
])
def test_bias_validation(loong_lib, buckets, status):
    assert ops.loong_rel_bias_check(_desc(), buckets.struct()) == status
    assert (ops.loong_attn_bias_workspace_size(_desc(), buckets.struct(), 1) > 0) == (status == ops.LOONG_OK)


def test_bias_descriptor_limits(loong_lib):
    b = ops.log_buckets(32, 128).struct()
    assert ops.loong_rel_bias_check(_desc(hq=3), b) == ops.LOONG_ERR_INVALID_ARG
    assert ops.loong_rel_bias_check(_desc(seqlen=1 << 30), b) == ops.LOONG_ERR_UNSUPPORTED
    assert ops.loong_rel_bias_check(_desc(softmax_scale=1e-9), b) == ops.LOONG_ERR_UNSUPPORTED
    assert ops.loong_rel_bias_check(_desc(softmax_scale=1e-3), b) == ops.LOONG_OK
    b.bounds = None
    assert ops.loong_rel_bias_check(_desc(), b) == ops.LOONG_ERR_INVALID_ARG
    assert ops.lib().loong_rel_bias_check(ctypes.byref(_desc()), None) == ops.LOONG_ERR_INVALID_ARG
    assert ops.loong_attn_bias_workspace_size(_desc(), ops.RelBuckets(1, []).struct(), 2) == 0


@pytest.mark.parametrize("causal", [1, 0])
@pytest.mark.parametrize("mode", [ops.MODE_FUSED, ops.MODE_STEPWISE])
def test_bias_workspace_sizes(loong_lib, causal, mode):
    up = lambda x: (x + 255) // 256 * 256
    d = _desc(causal=causal, mode=mode)
    b = ops.log_buckets(32, 128, causal=bool(causal))
    length = W.seqlen + 384 if causal else 2 * W.seqlen + 256
    lut = up(4 * W.hq * length) + up(length) + 2 * up(4 * length)
    assert ops.loong_attn_bias_workspace_size(d, b.struct(), 0) == \
        up(ops.loong_attn_workspace_size(d, 0)) + lut + up(1216 * 4)
    width = (W.hq // W.hkv) * (b.num_bounds + 1)
    part = up(4 * 16 * width * W.hkv * (W.seqlen // 128))
    assert ops.loong_attn_bias_workspace_size(d, b.struct(), 1) == \
        up(ops.loong_attn_workspace_size(d, 1)) + lut + part + 256 + up(8 * 64 * W.hkv * width)


def test_bias_calls_refuse_before_any_cuda_call(loong_lib):
    L, d, p = ops.lib(), _desc(), ctypes.c_void_p(PTR)
    bias = ops.log_buckets(32, 128).struct()
    bias.table = PTR
    big = 1 << 40
    fwd = lambda *a, ws=p, n=big: L.loong_attn_bias_fwd(ctypes.byref(d), ctypes.byref(bias), *a, ws, n, None)
    bwd = lambda *a, ws=p, n=big: L.loong_attn_bias_bwd(ctypes.byref(d), ctypes.byref(bias), *a, ws, n, None)
    odd = ctypes.c_void_p(PTR + 8)
    for i in range(5):
        for bad in (None, odd):
            assert fwd(*[bad if j == i else p for j in range(6)]) == ops.LOONG_ERR_INVALID_ARG
    assert fwd(p, p, p, p, p, odd) == ops.LOONG_ERR_INVALID_ARG          # o_res
    for i in [0, 1, 2, 3, 5, 6, 7, 8, 9, 10]:
        assert bwd(*[None if j == i else p for j in range(11)]) == ops.LOONG_ERR_INVALID_ARG
    need = ops.loong_attn_bias_workspace_size(d, bias, 0)
    for ws, n in ((None, big), (p, need - 1), (odd, big)):
        assert fwd(*[p] * 6, ws=ws, n=n) == ops.LOONG_ERR_WORKSPACE
    need = ops.loong_attn_bias_workspace_size(d, bias, 1)
    for ws, n in ((None, big), (p, need - 1), (odd, big)):
        assert bwd(*[p] * 11, ws=ws, n=n) == ops.LOONG_ERR_WORKSPACE
    bias.table = None
    assert fwd(*[p] * 6) == ops.LOONG_ERR_INVALID_ARG
    assert bwd(*[p] * 11) == ops.LOONG_ERR_INVALID_ARG


@pytest.mark.parametrize("n,m", [(2, 2), (4, 8), (7, 30), (8, 64), (32, 128), (32, 8192), (64, 1000), (128, 100000)])
def test_log_buckets_follow_their_definition(n, m):
    e, b = n // 2, ops.log_buckets(n, m)

    def bucket(x):
        if x < e:
            return x
        t = 0
        while t + 1 < n - e and x ** (n - e) * e ** (t + 1) >= m ** (t + 1) * e ** (n - e):
            t += 1
        return e + t
    for x in sorted(set(range(200)) | {m - 1, m, m + 1, m // 2, 10 * m}):
        assert b.bucket_of[sum(y <= x for y in b.bounds)] == bucket(x), x
    if n % 2 == 0:
        two = ops.log_buckets(2 * n, m, causal=False)
        for x in range(300):
            assert two.bucket_of[sum(y <= x for y in two.bounds)] == bucket(x)
            if x:
                assert two.bucket_of[sum(y <= -x for y in two.bounds)] == n + bucket(x)
    assert b.bounds == sorted(set(b.bounds)) and len(b.bucket_of) == len(b.bounds) + 1


def test_log_buckets_refusals():
    for bad in ((1, 8, True), (33, 8, False), (2, 8, False), (32, 16, True)):
        with pytest.raises(ValueError):
            ops.log_buckets(*bad)
    with pytest.raises(ValueError):
        ops.RelBuckets(3, [1, 2], [0, 1])
    with pytest.raises(ValueError):
        ops.RelBuckets(2, [2 ** 31])


def test_tensor_calls_refuse_wrong_tensors(loong_lib):
    x = inputs.make_inputs(W)
    buckets = ops.log_buckets(32, 128)
    table = torch.zeros((32, W.hq), dtype=torch.bfloat16)
    good = dict(q=x["q"], k=x["k"], v=x["v"], table=table)
    for n, t in (("q", x["q"][:, :-8]), ("k", x["k"].float()), ("v", x["v"].transpose(1, 2)), ("table", table.float()),
                 ("table", table[:16]), ("table", table.t())):
        with pytest.raises(ValueError):
            ops.attn_bias_fwd(W, **{**good, n: t}, buckets=buckets)
    with pytest.raises(ValueError, match="CUDA"):
        ops.attn_bias_fwd(W, **good, buckets=buckets)          # tensors on the CPU
    with pytest.raises(ops.LoongError):
        ops.attn_bias_fwd(W, **good, buckets=ops.RelBuckets(0, []))
