"""Host-side checks of the norm-and-rotation pass: refusals before any CUDA call
and the workspace size."""
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


def _opts(**kw):
    o = ops.make_qk_opts(64).struct()
    for k, v in kw.items():
        setattr(o, k, v)
    return o


@pytest.mark.parametrize("field,value", [
    ("rot_dim", 24), ("rot_dim", 80), ("rot_dim", -16), ("norm", 2), ("interleaved", -1), ("eps", -1e-6),
    ("eps", float("nan")), ("eps", float("inf")), ("w_offset", float("nan")), ("rot_scale", float("inf")),
    ("rot_base", 0.0), ("rot_base", float("inf")), ("q_stride", 128), ("q_stride", 260), ("k_stride", -8),
    ("dv_stride", 64), ("v_stride", (1 << 31) + 8)])
def test_options_refused(loong_lib, field, value):
    L, p, d = ops.lib(), ctypes.c_void_p(PTR), _desc()
    o = _opts(**{field: value})
    assert L.loong_qk_norm_rope_fwd(ctypes.byref(d), ctypes.byref(o), p, p, p, p, p, None, p, p, p, None) == \
        ops.LOONG_ERR_INVALID_ARG
    assert ops.loong_qk_norm_rope_bwd_workspace_size(d, o) == 0
    assert ops.loong_qk_norm_rope_bwd_workspace_size(d, _opts()) > 0
    assert ops.loong_qk_norm_rope_bwd_workspace_size(d, _opts(norm=0)) == 0


def test_frequencies_refused(loong_lib):
    bad = ops.make_qk_opts(64, inv_freq=[1.0] * 31 + [float("nan")]).struct()
    assert ops.loong_qk_norm_rope_bwd_workspace_size(_desc(), bad) == 0
    with pytest.raises(ValueError):
        ops.make_qk_opts(64, inv_freq=[1.0] * 31)


def test_calls_refuse_before_any_cuda_call(loong_lib):
    L, d, p, odd = ops.lib(), _desc(), ctypes.c_void_p(PTR), ctypes.c_void_p(PTR + 8)
    o = _opts()
    # q, k, v, wq, wk, positions, q_out, k_out, v_out
    fwd = lambda **b: L.loong_qk_norm_rope_fwd(ctypes.byref(d), ctypes.byref(o), *[b.get(n, p) for n in (
        "q", "k", "v", "wq", "wk", "positions", "q_out", "k_out", "v_out")], None)
    for n in ("q", "k", "q_out", "k_out", "v", "v_out"):          # v alone or v_out alone
        assert fwd(**{n: None}) == ops.LOONG_ERR_INVALID_ARG
    for n in ("q", "wq", "wk", "v_out"):
        assert fwd(**{n: odd}) == ops.LOONG_ERR_INVALID_ARG
    assert fwd(positions=ctypes.c_void_p(PTR + 4)) == ops.LOONG_ERR_INVALID_ARG
    names = ("q", "k", "wq", "wk", "positions", "dq_out", "dk_out", "dv_out", "dq", "dk", "dv", "dwq", "dwk", "ws")
    bwd = lambda n=1 << 40, o=o, **b: L.loong_qk_norm_rope_bwd(ctypes.byref(d), ctypes.byref(o),
                                                             *[b.get(x, p) for x in names], n, None)
    for n in ("q", "k", "dq_out", "dk_out", "dq", "dk", "dv", "dv_out"):
        assert bwd(**{n: None}) == ops.LOONG_ERR_INVALID_ARG
    assert bwd(o=_opts(norm=0)) == ops.LOONG_ERR_INVALID_ARG     # a weight gradient without a norm
    need = ops.loong_qk_norm_rope_bwd_workspace_size(d, o)
    assert bwd(n=need - 1) == ops.LOONG_ERR_WORKSPACE
    assert bwd(ws=None) == ops.LOONG_ERR_WORKSPACE
    assert bwd(ws=odd) == ops.LOONG_ERR_WORKSPACE
    assert bwd(dwq=ctypes.c_void_p(PTR + 2)) == ops.LOONG_ERR_INVALID_ARG


def test_tensor_calls_refuse_wrong_tensors(loong_lib):
    x = inputs.make_inputs(W)
    opts = ops.make_qk_opts(64)
    w1 = torch.ones(64)
    for kw in (dict(q=x["q"].transpose(1, 2)), dict(k=x["k"].float()), dict(wq=w1[:32]), dict(wk=w1.double()),
               dict(positions=torch.zeros((1, 1024), dtype=torch.int32)),
               dict(positions=torch.zeros((1, 1023), dtype=torch.int64)), dict(v=x["v"][..., ::2])):
        with pytest.raises(ValueError):
            ops.qk_norm_rope(W, opts, **{**dict(q=x["q"], k=x["k"], v=x["v"]), **kw})
    with pytest.raises(ValueError, match="CUDA"):
        ops.qk_norm_rope(W, opts, x["q"], x["k"], x["v"])
    with pytest.raises(ValueError, match="CUDA"):
        ops.qk_norm_rope_bwd(W, opts, x["q"], x["k"], x["q"], x["k"], x["v"])
    with pytest.raises(ValueError, match="into"):
        ops.qk_norm_rope_bwd(W, opts, x["q"], x["k"], x["q"], x["k"], x["v"], into=(x["q"], x["k"], None))
    with pytest.raises(ValueError):
        ops.qk_norm_rope_bwd(W, opts, x["q"], x["k"], x["q"], x["k"][:, 1:], x["v"])


# batch, tokens of the view that is expanded to it
@pytest.mark.parametrize("batch,seqlen,b,s", [(1, 64, 1, 1), (2, 64, 1, 1), (8, 1, 1, 1), (2, 64, 1, 64)])
def test_expanded_projections_refused(loong_lib, batch, seqlen, b, s):
    """One token's (or one sequence's) memory repeated over a shape: the call
    would read, and through ``into`` write, as if every token had its own."""
    w = inputs.small(seqlen, 4, 2, 64, placement=0).with_(batch=batch)
    full = lambda h: torch.zeros((batch, seqlen, h, 64), dtype=torch.bfloat16)
    repeated = lambda h: torch.zeros((b, s, h, 64), dtype=torch.bfloat16).expand(batch, seqlen, h, 64)
    good, opts = [full(4), full(2), full(2)], ops.make_qk_opts(64)
    for i, heads in enumerate((4, 2, 2)):
        bad = list(good)
        bad[i] = repeated(heads)
        with pytest.raises(ValueError, match="evenly spaced tokens"):
            ops._token_strides("qkv", bad, w, bad[0].device)
        with pytest.raises(ValueError, match="evenly spaced tokens"):
            ops.qk_norm_rope(w, opts, *bad)
    assert ops._token_strides("qkv", good, w, good[0].device) == [256, 128, 128]


def test_overlapping_tokens_refused(loong_lib):
    """A token's stride below its own elements."""
    w = inputs.small(64, 4, 2, 64, placement=0)
    q = torch.zeros(65 * 256, dtype=torch.bfloat16).as_strided((1, 64, 4, 64), (0, 248, 64, 1))
    with pytest.raises(ValueError, match="evenly spaced tokens"):
        ops._token_strides("q", [q], w, q.device)


def test_expanded_gradients_refused(loong_lib, monkeypatch):
    """The same for the projections' gradients, which the call writes."""
    w = inputs.small(64, 4, 2, 64, placement=0)
    full = [torch.zeros((1, 64, h, 64), dtype=torch.bfloat16) for h in (4, 2, 2)]
    monkeypatch.setattr(ops, "_on", lambda device, stream: (ops._NOTHING, 0))    # past the device's check
    launched = []
    monkeypatch.setattr(ops, "loong_qk_norm_rope_bwd", lambda *a: launched.append(a))
    for i in range(3):
        into = list(full)
        into[i] = full[i][:, :1].expand(1, 64, -1, 64)
        with pytest.raises(ValueError, match="evenly spaced tokens"):
            ops.qk_norm_rope_bwd(w, ops.make_qk_opts(64), *full[:2], *full, into=into)
    assert not launched


def test_stream_numbers(monkeypatch):
    """A number stands for the stream of that handle, on the tensors' device."""
    import contextlib
    entered = []

    class Stream:
        def __init__(self, handle, device):
            self.cuda_stream, self.device = handle, device

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: entered.append(s) or contextlib.nullcontext(s.device))
    device = torch.device("cuda:0")
    for number, handle in ((0x7f00, 0x7f00), (0, 0), (1, 0), (2, 2)):
        where, stream = ops._on(device, number)
        with where:
            assert entered[-1] is stream and stream.cuda_stream == handle and stream.device == device


def test_counting_positions_keep_one_struct():
    """A position that moves on with every call finds what is kept, and leaves the struct of an earlier call alone."""
    opts = ops.make_qk_opts(64)
    first = opts._struct_of((384, 384, 384), pos_begin=7)
    for pos in range(200):
        assert opts._struct_of((384, 384, 384), pos_begin=pos).pos_begin == pos
    assert first.pos_begin == 7 and len(opts._structs) == 1
    one = opts._struct_of((384, 384, 384), pos_begin=-3)
    for name, _ in ops.LoongQkOpts._fields_:
        if name not in ("pos_begin", "inv_freq"):
            assert getattr(one, name) == getattr(opts.struct((384, 384, 384)), name), name
    assert [one.inv_freq[i] for i in range(32)] == [10000.0 ** (-2.0 * i / 64) for i in range(32)]


def test_bases_whose_frequencies_are_infinite_refused(loong_lib):
    for base in (5e-324, 1e-309):
        assert ops.loong_qk_norm_rope_bwd_workspace_size(_desc(), ops.make_qk_opts(64, base=base).struct()) == 0
    for base in (2.0 ** -1022, 1.7e308):
        assert ops.loong_qk_norm_rope_bwd_workspace_size(_desc(), ops.make_qk_opts(64, base=base).struct()) > 0
