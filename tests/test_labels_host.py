"""Label-side operators, what needs no GPU: refusals at the C boundary and in the Python entry
points, workspace sizes, the descriptors of states."""
import ctypes

import pytest
import torch

import rnn_transducer_loss_gb300 as pkg
from rnn_transducer_loss_gb300 import _native as N
from rnn_transducer_loss_gb300 import beam
from rnn_transducer_loss_gb300 import build as B


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return N.load()


def embed(**kw):
    a = dict(weight=1 << 20, dt=N.RNNT_F32, V=10, D=8, weight_stride=8, tokens=4096,
             tokens_stride=5, lengths=None, B=2, S=5, has_start=0, start=0, scale=1.0,
             out=1 << 21, status_dev=None, stream=None)
    a.update(kw)
    return N.rnnt_embed(*a.values())


@pytest.mark.parametrize("bad", [
    dict(weight=None), dict(out=None), dict(tokens=None), dict(dt=3), dict(V=0), dict(D=0),
    dict(D=(1 << 20) + 1, weight_stride=1 << 25), dict(weight_stride=7), dict(tokens_stride=4),
    dict(B=0), dict(S=-1), dict(S=0), dict(B=1 << 20, S=1 << 12, tokens_stride=1 << 12),
    dict(has_start=1, start=10), dict(has_start=1, start=-11), dict(scale=float("nan")),
    dict(weight=(1 << 20) + 2), dict(out=(1 << 21) + 1), dict(out=(1 << 20) + 64),
], ids=str)
def test_embed_refuses(bad):
    assert embed(**bad) == N.RNNT_INVALID_VALUE


def embed_grad(**kw):
    a = dict(grad_out=1 << 20, dt=N.RNNT_F16, tokens=4096, tokens_stride=5, lengths=None, B=2, S=5,
             has_start=0, start=0, V=10, D=8, scale=1.0, grad_weight=1 << 21, workspace=1 << 22,
             workspace_bytes=1 << 30, status_dev=None, stream=None)
    a.update(kw)
    return N.rnnt_embed_grad(*a.values())


@pytest.mark.parametrize("bad", [
    dict(grad_out=None), dict(grad_weight=None), dict(tokens=None),
    dict(workspace=None, S=2100, tokens_stride=2100, grad_weight=1 << 24),
    dict(dt=-1), dict(V=0), dict(D=0), dict(B=0), dict(S=0), dict(tokens_stride=4),
    dict(has_start=1, start=10), dict(scale=float("nan")), dict(workspace=(1 << 22) + 64),
    dict(grad_out=(1 << 20) + 1), dict(grad_weight=(1 << 20) + 64), dict(D=(1 << 20) + 1),
], ids=str)
def test_embed_grad_refuses(bad):
    assert embed_grad(**bad) == N.RNNT_INVALID_VALUE


def test_embed_grad_workspace():
    assert N.rnnt_embed_grad_workspace_size(2, 2048, 0, 10, 8) == 0       # 4096 places: none
    n = N.rnnt_embed_grad_workspace_size(2, 2100, 0, 10, 8)
    assert n > 0 and n % 256 == 0
    assert embed_grad(workspace_bytes=n - 1, S=2100, tokens_stride=2100, grad_weight=1 << 24) \
        == N.RNNT_WORKSPACE_TOO_SMALL
    big = N.rnnt_embed_grad_workspace_size(64, 1023, 1, 50000, 1024)
    assert 65536 * 16 <= big <= 65536 * (16 + 4 * 1024 // 8)
    for args in ((0, 5, 0, 10, 8), (2, 0, 0, 10, 8), (2, 5, 0, 0, 8), (2, 5, 0, 10, 0),
                 (1 << 20, 1 << 12, 0, 10, 8)):
        with pytest.raises(N.RNNTError):
            N.rnnt_embed_grad_workspace_size(*args)


def select(**kw):
    a = dict(logits=1 << 20, dt=N.RNNT_F32, B=2, K=4, V=30, batch_stride=120, beam_stride=30,
             scores=4096, finished=None, Ko=4, fused=1, out_scores=8192, out_tokens=8448,
             out_parents=8704, workspace=1 << 21, workspace_bytes=1 << 30, status_dev=None,
             stream=None)
    a.update(kw)
    return N.rnnt_beam_select(*a.values())


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(scores=None), dict(out_scores=None), dict(out_tokens=None),
    dict(out_parents=None), dict(workspace=None, V=1 << 18), dict(dt=9), dict(B=0), dict(K=0), dict(K=65),
    dict(V=0), dict(V=(1 << 20) + 1), dict(Ko=0), dict(Ko=65), dict(batch_stride=-1),
    dict(beam_stride=-1), dict(logits=(1 << 20) + 2), dict(workspace=(1 << 21) + 16),
    dict(B=1 << 29),
], ids=str)
def test_select_refuses(bad):
    assert select(**bad) == N.RNNT_INVALID_VALUE


def test_select_workspace():
    assert N.rnnt_beam_workspace_size(2, 4, 30, 4, N.RNNT_F32) == 0        # one launch: none
    n = N.rnnt_beam_workspace_size(2, 4, 1 << 18, 4, N.RNNT_F32)
    assert n > 0 and n % 256 == 0
    assert select(V=1 << 18, workspace_bytes=n - 1) == N.RNNT_WORKSPACE_TOO_SMALL
    assert N.rnnt_beam_workspace_size(2, 4, 1 << 20, 8, N.RNNT_F32) > n
    for args in ((0, 4, 30, 4, 0), (2, 65, 30, 4, 0), (2, 4, 30, 0, 0), (2, 4, 30, 4, 3)):
        with pytest.raises(N.RNNTError):
            N.rnnt_beam_workspace_size(*args)


def reorder(parents=4096, B=2, K=3, Ko=3, n_states=1, n=(1, 1, 1), **kw):
    s = N.State()
    s.src, s.dst, s.row_bytes = 1 << 20, 1 << 21, 64
    s.src_batch = s.dst_batch = 192
    s.src_beam = s.dst_beam = 64
    for i in range(3):
        s.n[i] = n[i]
    for k, v in kw.items():
        if isinstance(v, tuple):
            for i in range(3):
                getattr(s, k)[i] = v[i]
        else:
            setattr(s, k, v)
    return N.rnnt_beam_reorder(ctypes.byref(s), n_states, parents, B, K, Ko, None, None)


@pytest.mark.parametrize("bad", [
    dict(parents=None), dict(B=0), dict(K=0), dict(Ko=0), dict(n_states=0), dict(n_states=17),
    dict(src=None), dict(dst=None), dict(row_bytes=0), dict(n=(0, 1, 1)),
    dict(n=(2, 1, 1), src_stride=(-8, 0, 0)), dict(src_beam=-64), dict(dst_batch=-1),
    dict(dst=1 << 20), dict(dst=(1 << 20) + 128),
    dict(n=(1 << 30, 1 << 30, 1 << 30)), dict(n=(2, 1, 1)), dict(dst_beam=0), dict(dst_batch=0),
], ids=str)
def test_reorder_refuses(bad):
    assert reorder(**bad) == N.RNNT_INVALID_VALUE


def test_state_layout():
    assert ctypes.sizeof(N.State) == 8 * 3 + 16 + 24 * 2 + 8 * 4
    assert N.State.src_stride.offset == 40


@pytest.mark.parametrize("shape,view,d,row,axes", [
    ((3, 4, 7), None, 0, 28, []),
    ((2, 3, 4, 10), None, 1, 40, [(2, 480)]),
    ((3, 4, 5, 9, 8), (Ellipsis, slice(0, 6), slice(None)), 0, 192, [(5, 288)]),
    ((3, 4, 5, 9, 8), (Ellipsis, slice(0, 6)), 0, 24, [(45, 32)]),
    ((2, 6, 3, 4, 8), None, 2, 32, [(12, 384)]),
    ((3, 4), None, 0, 4, []),
    ((3, 4, 6, 1), None, 0, 24, []),
])
def test_describe(shape, view, d, row, axes):
    x = torch.zeros(shape)
    x = x if view is None else x[view]
    y = torch.empty(x.shape)
    got = beam._describe(tuple(x.shape), x.stride(), y.stride(), 4, d)
    assert got[0] == row
    assert [(n, a) for n, a in zip(got[1], got[2]) if n > 1] == axes
    assert got[4:] == (x.stride(d) * 4, x.stride(d + 1) * 4, y.stride(d) * 4, y.stride(d + 1) * 4)
    s = N.State.from_buffer_copy(beam._POINTERS.pack(64, 128) + beam._pack(got))
    assert (s.src, s.dst, s.row_bytes, s.n[0], s.dst_beam) == (64, 128, row, got[1][0], got[7])


def test_describe_refuses_many_axes():
    x = torch.zeros(2, 3, 5, 5, 5, 5, 5)[:, :, ::2, ::2, ::2, ::2, ::2]
    with pytest.raises(ValueError):
        beam._describe(tuple(x.shape), x.stride(), torch.empty(x.shape).stride(), 4, 0)


def test_python_refuses():
    """No CUDA tensor, no call: argument checks that come first."""
    w, tok = torch.zeros(4, 8), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.rnnt_embed(w, tok)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.rnnt_embed_grad(torch.zeros(2, 3, 8), tok, 4)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.rnnt_beam_select(torch.zeros(2, 3, 8), torch.zeros(2, 3))
    with pytest.raises(ValueError, match="CUDA"):
        pkg.rnnt_beam_reorder([torch.zeros(2, 3)], tok)
    assert pkg.RNNTEmbedding(5, 3, start=0).weight.shape == (5, 3)
    with pytest.raises(AttributeError):
        pkg.no_such_name
