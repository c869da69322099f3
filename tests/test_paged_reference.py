"""CPU: the definitions that the calls over a paged cache are tested against, and the calls' refusals."""

import ctypes

import numpy as np
import pytest
import torch

import paged_reference as ref


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_60_gb300 import build

    build.build()
    import speculative_decoding_verification_60_gb300 as svp

    return svp.load()


def test_paths():
    parent = [-1, 0, 0, 1, 3, 2]
    assert ref.is_tree(parent) and not ref.is_tree([0, 0]) and not ref.is_tree([-1, 1]) and not ref.is_tree([-1, -1])
    assert ref.path(parent, 4) == [0, 1, 3, 4] and ref.path(parent, 0) == [0]


def test_turn_keeps_lengths_and_differences():
    """Turned heads keep their lengths, and a product depends on the difference of positions only."""
    g = torch.Generator().manual_seed(0)
    x, y = torch.randn(3, 1, 16, generator=g).double(), torch.randn(3, 1, 16, generator=g).double()
    f = torch.tensor([1.0, 0.1, 0.01, 0.001])
    for pairs in (False, True):
        at = torch.tensor([5, 70, 900])
        a, b = ref.turn(x, at, f, pairs), ref.turn(y, at + 3, f, pairs)
        c, d = ref.turn(x, at * 0, f, pairs), ref.turn(y, at * 0 + 3, f, pairs)
        # f is held in 32 bits and its products are exact in 64 to 2^-53 of the angle
        assert torch.allclose((a * b).sum(2), (c * d).sum(2), atol=1e-11)
        assert torch.allclose(a.square().sum(2), x.square().sum(2))


def test_attend_is_a_mean():
    """Equal keys: the mean of the values that a node sees."""
    k, v = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16), torch.arange(8.0).view(2, 4, 1, 1).expand(2, 4, 1, 64).bfloat16()
    table = torch.tensor([[1, 0]], dtype=torch.int32)
    out, _ = ref.attend(torch.ones(1, 3, 1, 64).bfloat16(), k, v, table, torch.tensor([4]),
                        torch.tensor([-1, 0, 0], dtype=torch.int32))
    # sequence 4 5 6 7, nodes 0 1 2
    assert torch.allclose(out[0, :, 0, 0], torch.tensor([22 / 5, 23 / 6, 24 / 6], dtype=torch.float64))


def test_adjust_by_hand():
    x = np.array([2.0, -2.0, 1.0, 0.0])
    y = ref.adjust(x, 0, 1, np.array([[0, 1, 1]]), [3], [1], np.array([[9, 2]]), [-1, 0], [2.0], [0.5], [0.25],
                   np.array([[3, 3, -1]]), np.array([[1.0, 2.0, 9.0]]), np.array([[[15], [15]]]))
    assert np.allclose(y, [1.0, -4.0 - 1.25, 0.5 - 0.75, 3.0])


def test_keep_by_hand():
    cache = np.arange(8).reshape(2, 4, 1)
    assert ref.keep(cache, np.array([[0, 2, 3]]), [2], [1], np.array([[1, 0]])) == []
    assert cache[:, :, 0].tolist() == [[0, 1, 2, 3], [4, 5, 7, 0]]


def _status(lib, name, good, **change):
    args = dict(good, **change)
    return getattr(lib, name)(*args.values())


def _layout(**change):
    from speculative_decoding_verification_60_gb300 import CacheLayout

    return ctypes.byref(CacheLayout(**dict(dict(blocks=4, page_size=16, heads=2, dim=64, block_stride=2048,
                                                entry_stride=128, head_stride=64), **change)))


def test_append_refusals(lib):
    d = ctypes.c_void_p(4096)
    good = dict(q=d, k=d, v=d, dtype=0, T=2, heads=4, qt=512, qh=64, kt=512, kh=64, vt=512, vh=64, qn=None, kn=None,
                eps=1e-6, pos=d, inv=d, rot=64, inter=0, slots=d, out=d, kc=d, vc=d, layout=_layout(), err=None,
                stream=None)
    bad = lambda **k: _status(lib, "spec_append_kv", good, **k)  # noqa: E731
    for change in (dict(k=None), dict(v=None), dict(dtype=1), dict(T=-1), dict(heads=0), dict(slots=None), dict(out=None),
                   dict(kc=None), dict(vc=None), dict(pos=None), dict(inv=None), dict(rot=66), dict(rot=-2), dict(rot=3),
                   dict(qn=d), dict(kn=d), dict(q=None, qn=d, kn=d), dict(eps=float("nan")), dict(eps=-1.0),
                   dict(layout=None), dict(layout=_layout(blocks=0)), dict(layout=_layout(page_size=0)),
                   dict(layout=_layout(entry_stride=-1))):
        assert bad(**change) == 1, change
    for change in (dict(rot=4), dict(layout=_layout(dim=60), rot=0), dict(layout=_layout(dim=264)), dict(qt=513),
                   dict(k=ctypes.c_void_p(4100)), dict(layout=_layout(head_stride=66))):
        assert bad(**change) == 2, change
    assert bad(T=0) == 0


def test_attention_refusals(lib):
    d = ctypes.c_void_p(4096)
    need = lib.spec_tree_attention_workspace(2, 5, 4, 2, 64)
    assert need > 0 and lib.spec_tree_attention_workspace(0, 5, 4, 2, 64) == 0
    good = dict(q=d, dtype=0, B=2, N=5, heads=4, qr=1280, qn=256, qh=64, k=d, v=d, layout=_layout(), table=d, M=4, step=4,
                lens=d, parent=None, pstep=0, counts=None, scale=0.1, out=d, err=None, ws=d, bytes=need, stream=None)
    bad = lambda **k: _status(lib, "spec_tree_attention", good, **k)  # noqa: E731
    for change in (dict(q=None), dict(dtype=1), dict(B=0), dict(N=0), dict(heads=3), dict(heads=0), dict(qr=-8),
                   dict(k=None), dict(v=None), dict(layout=None), dict(table=None), dict(M=0), dict(step=3),
                   dict(lens=None), dict(parent=d, pstep=4), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                   dict(scale=float("inf")), dict(scale=3e38), dict(out=None)):
        assert bad(**change) == 1, change
    for change in (dict(N=1025), dict(B=65536), dict(heads=258), 
                   dict(M=2**31 - 1, step=2**31 - 1, layout=_layout(page_size=1024, block_stride=2**17)), dict(layout=_layout(dim=136)),
                   dict(layout=_layout(dim=68)), dict(qn=260), dict(k=ctypes.c_void_p(4104)),
                   dict(q=ctypes.c_void_p(4104)), dict(layout=_layout(entry_stride=132))):
        assert bad(**change) == 2, change
    for change in (dict(ws=None), dict(bytes=need - 1), dict(ws=ctypes.c_void_p(4096 + 128))):
        assert bad(**change) == 3, change


def test_adjust_refusals(lib):
    from speculative_decoding_verification_60_gb300 import Adjustments

    d = 4096
    p = ctypes.c_void_p(d)
    make = lambda **k: ctypes.byref(Adjustments(**k))  # noqa: E731
    good = dict(x=p, dtype=0, B=2, R=3, V=64, step=64, a=make(), out=p, ostep=64, err=None, stream=None)
    bad = lambda **k: _status(lib, "spec_adjust_logits", good, **k)  # noqa: E731
    for change in (dict(x=None), dict(dtype=2), dict(B=-1), dict(R=0), dict(V=0), dict(step=63), dict(a=None),
                   dict(out=None), dict(ostep=63), dict(step=65), dict(a=make(history=d, history_capacity=4, history_stride=4)),
                   dict(a=make(history=d, history_lens=d, history_capacity=4, history_stride=3)),
                   dict(a=make(history=d, history_lens=d, history_capacity=-1)), dict(a=make(drafted=d, drafted_stride=1)),
                   dict(a=make(parent=d, parent_stride=2)), dict(a=make(bias_ids=d, bias_count=1)),
                   dict(a=make(bias_ids=d, bias_values=d, bias_count=-1)), dict(a=make(allowed=d, allowed_stride=1))):
        assert bad(**change) == 1, change
    for change in (dict(V=524281, step=524281, ostep=524281), dict(R=1025), dict(B=65536),
                   dict(a=make(bias_ids=d, bias_values=d, bias_count=1025))):
        assert bad(**change) == 2, change
    assert bad(B=0) == 0


def test_keep_refusals(lib):
    d = ctypes.c_void_p(4096)
    two = (ctypes.c_void_p * 2)(4096, 8192)
    good = dict(planes=two, n=2, size=2, layout=_layout(), B=2, W=4, path=d, acc=d, lens=d, table=d, M=4, step=4, err=None,
                stream=None)
    bad = lambda **k: _status(lib, "spec_keep_path", good, **k)  # noqa: E731
    for change in (dict(planes=None), dict(n=-1), dict(size=3), dict(layout=None), dict(B=-1), dict(W=0), dict(path=None),
                   dict(acc=None), dict(lens=None), dict(table=None), dict(M=0), dict(step=3),
                   dict(planes=(ctypes.c_void_p * 2)(4096, None))):
        assert bad(**change) == 1, change
    assert bad(B=65536) == 2 and bad(W=1025) == 2
    assert bad(n=0) == 0 and bad(B=0) == 0


def test_bindings_refuse_what_the_calls_cannot_take(lib):
    import speculative_decoding_verification_60_gb300 as svp

    x = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        svp.tree_attention(x, x, x, torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        svp.tree_attention(x.float(), x, x, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        svp.append_kv(x[0], x[0], x[0], None, None, x, x)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        svp.append_kv(x[0].float(), x[0].float(), x[0].float(), None, None, x, x)
    with pytest.raises(ValueError, match="shape"):
        svp.adjust_logits(x[0, 0])
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        svp.adjust_logits(x[0].half())
    with pytest.raises(ValueError, match="CUDA"):
        svp.keep_path([x], torch.zeros(2, 4, dtype=torch.int32), None, None, None)
