"""Host-side checks of the masked and the paged attention: refusals before any
CUDA call, workspace sizes, and the range maker against its definition."""
import ctypes
import itertools

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


@pytest.mark.parametrize("cap,status", [
    (0.0, ops.LOONG_OK), (30.0, ops.LOONG_OK), (2.0 ** -20, ops.LOONG_OK), (2.0 ** 20, ops.LOONG_OK),
    (-1.0, ops.LOONG_ERR_INVALID_ARG), (float("nan"), ops.LOONG_ERR_INVALID_ARG),
    (float("inf"), ops.LOONG_ERR_INVALID_ARG), (2.0 ** -21, ops.LOONG_ERR_UNSUPPORTED),
    (2.0 ** 21, ops.LOONG_ERR_UNSUPPORTED),
])
def test_cap_validation(loong_lib, cap, status):
    m = ops.make_mask(None, cap)
    assert ops.loong_attn_mask_check(_desc(), m) == status
    for pass_ in (0, 1):
        assert (ops.loong_attn_mask_workspace_size(_desc(), m, pass_) > 0) == (status == ops.LOONG_OK)


def test_mask_descriptor_limits(loong_lib):
    m, capped = ops.make_mask(), ops.make_mask(None, 30.0)
    assert ops.loong_attn_mask_check(_desc(hq=3), m) == ops.LOONG_ERR_INVALID_ARG
    assert ops.loong_attn_mask_check(_desc(seqlen=(1 << 30) + 16, batch=1), m) == ops.LOONG_ERR_UNSUPPORTED
    assert ops.loong_attn_mask_check(_desc(hq=65536, hkv=65536, seqlen=16), m) == ops.LOONG_ERR_UNSUPPORTED
    assert ops.loong_attn_mask_check(_desc(softmax_scale=1e-9), m) == ops.LOONG_OK
    assert ops.loong_attn_mask_check(_desc(softmax_scale=1e-9), capped) == ops.LOONG_ERR_UNSUPPORTED
    assert ops.loong_attn_mask_check(_desc(softmax_scale=1e9), capped) == ops.LOONG_ERR_UNSUPPORTED
    assert ops.lib().loong_attn_mask_check(ctypes.byref(_desc()), None) == ops.LOONG_ERR_INVALID_ARG
    assert ops.lib().loong_attn_mask_check(None, ctypes.byref(m)) == ops.LOONG_ERR_INVALID_ARG
    assert ops.loong_attn_mask_workspace_size(_desc(), m, 2) == 0


@pytest.mark.parametrize("mode", [ops.MODE_FUSED, ops.MODE_STEPWISE])
@pytest.mark.parametrize("seqlen", [1024, 1040])
def test_mask_workspace_sizes(loong_lib, mode, seqlen):
    up = lambda x: (x + 255) // 256 * 256
    m = ops.make_mask()
    one = dict(cp=1, hp=1, ring_inner=1, ring_outer=1, placement=ops.PLACEMENT_CONTIGUOUS)
    for layout in (ops.LAYOUT_NATURAL, ops.LAYOUT_RANK_MAJOR):
        d = _desc(mode=mode, seqlen=seqlen, layout=layout)
        whole = mode == ops.MODE_FUSED and layout == ops.LAYOUT_NATURAL   # the sequence is one block
        base = _desc(mode=mode, seqlen=seqlen, **one) if whole else d
        tiles = -(-seqlen // 128) if whole else 8 * -(-(seqlen // 8) // 128)
        assert ops.loong_attn_mask_workspace_size(d, m, 0) == \
            up(ops.loong_attn_workspace_size(base, 0)) + up(16 * tiles) + up(4 * 1216) + up(4)
        # 16 key tiles' blocks for 152 SMs: the two query heads of a group go to two, each with a part of dK and dV
        parts = 2 * up(2 * 4 * seqlen * W.hkv * W.head_dim) if mode == ops.MODE_FUSED else 0
        assert ops.loong_attn_mask_workspace_size(d, m, 1) == \
            up(ops.loong_attn_workspace_size(base, 1)) + up(16 * tiles) + up(tiles * W.hq) + parts


def test_mask_calls_refuse_before_any_cuda_call(loong_lib):
    L, d, m = ops.lib(), ctypes.byref(_desc()), ctypes.byref(ops.make_mask())
    n = ops.loong_attn_mask_workspace_size(_desc(), ops.make_mask(), 0)
    for bad in range(5):
        a = [PTR] * 5
        for value in (None, PTR + 4):
            a[bad] = value
            assert L.loong_attn_mask_fwd(d, m, *a, None, PTR, n, None) == ops.LOONG_ERR_INVALID_ARG
    assert L.loong_attn_mask_fwd(d, m, *[PTR] * 5, None, PTR, n - 1, None) == ops.LOONG_ERR_WORKSPACE
    assert L.loong_attn_mask_fwd(d, m, *[PTR] * 5, None, None, n, None) == ops.LOONG_ERR_WORKSPACE
    assert L.loong_attn_mask_fwd(d, m, *[PTR] * 5, PTR + 2, PTR, n, None) == ops.LOONG_ERR_INVALID_ARG
    odd = ops.make_mask()
    odd.key_range = PTR + 4
    assert L.loong_attn_mask_fwd(d, ctypes.byref(odd), *[PTR] * 5, None, PTR, n, None) == ops.LOONG_ERR_INVALID_ARG
    n = ops.loong_attn_mask_workspace_size(_desc(), ops.make_mask(), 1)
    for bad in range(10):
        a = [PTR] * 10   # q k v o o_res lse dout dq dk dv
        a[bad] = PTR + 4
        assert L.loong_attn_mask_bwd(d, m, *a, PTR, n, None) == ops.LOONG_ERR_INVALID_ARG
        if bad != 4:
            a[bad] = None
            assert L.loong_attn_mask_bwd(d, m, *a, PTR, n, None) == ops.LOONG_ERR_INVALID_ARG
    assert L.loong_attn_mask_bwd(d, m, *[PTR] * 10, PTR, n - 1, None) == ops.LOONG_ERR_WORKSPACE


PAGED = dict(batch=3, tokens=10, hq=8, hkv=2, head_dim=128, page_size=64, num_pages=100, max_pages=30, window=0,
             softmax_scale=0.0, score_cap=0.0, q_stride=0, k_stride=0, v_stride=0)


@pytest.mark.parametrize("change,status", [
    ({}, ops.LOONG_OK), ({"tokens": 0}, ops.LOONG_OK), ({"window": 1}, ops.LOONG_OK), ({"score_cap": 30.0}, ops.LOONG_OK),
    ({"q_stride": 1536, "k_stride": 1536, "v_stride": 256}, ops.LOONG_OK),
    ({"batch": 0}, ops.LOONG_ERR_INVALID_ARG), ({"tokens": -1}, ops.LOONG_ERR_INVALID_ARG),
    ({"hq": 9}, ops.LOONG_ERR_INVALID_ARG), ({"hkv": 0}, ops.LOONG_ERR_INVALID_ARG),
    ({"num_pages": 0}, ops.LOONG_ERR_INVALID_ARG), ({"max_pages": 0}, ops.LOONG_ERR_INVALID_ARG),
    ({"window": -1}, ops.LOONG_ERR_INVALID_ARG), ({"page_size": 0}, ops.LOONG_ERR_INVALID_ARG),
    ({"q_stride": 1016}, ops.LOONG_ERR_INVALID_ARG), ({"k_stride": 260}, ops.LOONG_ERR_INVALID_ARG),
    ({"v_stride": -8}, ops.LOONG_ERR_INVALID_ARG), ({"v_stride": (1 << 31) + 8}, ops.LOONG_ERR_INVALID_ARG),
    ({"softmax_scale": float("nan")}, ops.LOONG_ERR_INVALID_ARG), ({"score_cap": -2.0}, ops.LOONG_ERR_INVALID_ARG),
    ({"head_dim": 96}, ops.LOONG_ERR_UNSUPPORTED), ({"page_size": 48}, ops.LOONG_ERR_UNSUPPORTED),
    ({"page_size": 4}, ops.LOONG_ERR_UNSUPPORTED), ({"page_size": 2048}, ops.LOONG_ERR_UNSUPPORTED),
    ({"hq": 258, "hkv": 2}, ops.LOONG_ERR_UNSUPPORTED), ({"batch": 4097}, ops.LOONG_ERR_UNSUPPORTED),
    ({"num_pages": 1 << 24}, ops.LOONG_ERR_UNSUPPORTED), ({"max_pages": (1 << 24) + 1}, ops.LOONG_ERR_UNSUPPORTED),
    ({"score_cap": 2.0 ** 21}, ops.LOONG_ERR_UNSUPPORTED),
    ({"score_cap": 30.0, "softmax_scale": 1e-9}, ops.LOONG_ERR_UNSUPPORTED),
    # units of work that pass 32 bits
    ({"batch": 4096, "max_pages": 1 << 24}, ops.LOONG_ERR_UNSUPPORTED),
])
def test_paged_validation(loong_lib, change, status):
    d = ops.LoongPagedDesc(**(PAGED | change))
    assert ops.loong_paged_check(d) == status
    assert (ops.loong_paged_attn_workspace_size(d) > 0) == (status == ops.LOONG_OK)


def test_paged_calls_refuse_before_any_cuda_call(loong_lib):
    L, d = ops.lib(), ops.LoongPagedDesc(**PAGED)
    n = ops.loong_paged_attn_workspace_size(d)
    call = lambda a, ws=PTR, nbytes=n: L.loong_paged_attn(ctypes.byref(d), *a, ws, nbytes, None)
    full = [PTR] * 10   # q k v k_pages v_pages table lens starts o lse
    for i in range(10):
        a = list(full)
        a[i] = None     # k or v alone, or a pointer that is needed
        assert call(a) == ops.LOONG_ERR_INVALID_ARG, i
        a[i] = PTR + 2
        assert call(a) == ops.LOONG_ERR_INVALID_ARG, i
    assert call(full, nbytes=n - 1) == ops.LOONG_ERR_WORKSPACE
    assert call(full, ws=None) == ops.LOONG_ERR_WORKSPACE
    d.tokens = 0
    assert call([None] * 10, None, 0) == ops.LOONG_OK
    assert L.loong_paged_attn(None, *full, PTR, n, None) == ops.LOONG_ERR_INVALID_ARG


def test_paged_workspace_covers_every_block(loong_lib):
    """Each of the 152 blocks stores up to two shares of 128 or 256 rows."""
    for change in ({}, {"tokens": 5000}, {"head_dim": 64}, {"hq": 2}):
        d = ops.LoongPagedDesc(**(PAGED | change))
        slots = 2 if d.tokens * (d.hq // d.hkv) > 128 * d.batch else 1
        assert ops.loong_paged_attn_workspace_size(d) >= 152 * 2 * slots * 128 * (d.head_dim + 4) * 4


@pytest.mark.parametrize("causal,window,prefix", [(True, 0, False), (True, 3, False), (True, 0, True), (False, 0, False),
                                                  (False, 2, False)])
def test_document_ranges(causal, window, prefix):
    lengths, s = [[4, 1, 0, 5], [], [12]], 12
    pre = [[2, 9, 0, 5], [], [1]] if prefix else None
    r = ops.document_ranges(lengths, s, prefix=pre, window=window, causal=causal)
    assert r.shape == (3, s, 2) and r.dtype == torch.int32
    for b, docs in enumerate(lengths):
        owner = list(itertools.chain(*([i] * n for i, n in enumerate(docs))))
        start = [sum(docs[:i]) for i in range(len(docs))]
        for i in range(s):
            want = set()
            for j in range(s):
                if i >= len(owner) or j >= len(owner) or owner[i] != owner[j]:
                    continue
                near = not window or (i - window < j if causal else abs(i - j) <= window)
                sees = j <= i if causal else True
                if prefix:
                    sees |= j - start[owner[i]] < pre[b][owner[i]]
                if near and sees:
                    want.add(j)
            assert set(range(*r[b, i].tolist())) == want, (b, i)


def test_document_ranges_refuses():
    with pytest.raises(ValueError, match="do not fit"):
        ops.document_ranges([[5, 6]], 10)
    with pytest.raises(ValueError, match="do not fit"):
        ops.document_ranges([[-1]], 10)
    with pytest.raises(ValueError, match="prefix"):
        ops.document_ranges([[5]], 10, prefix=[[1, 2]])
    with pytest.raises(ValueError, match="prefix"):
        ops.document_ranges([[5]], 10, prefix=[[1]], window=3)
    with pytest.raises(ValueError, match="window"):
        ops.document_ranges([[5]], 10, window=-3)


def test_tensors_off_the_gpu_are_refused(loong_lib):
    x = inputs.make_inputs(W)
    with pytest.raises(ValueError, match="CUDA device"):
        ops.attn_mask_fwd(W, x["q"], x["k"], x["v"])
    pages = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        ops.paged_attn(x["q"][0, :1], pages, pages, torch.zeros(1, 4, dtype=torch.int32), one,
                       torch.zeros(2, dtype=torch.int32))
