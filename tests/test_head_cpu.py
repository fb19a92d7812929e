"""Argument checks of the layer norm and cross entropy calls: they come before any CUDA call, so they are
testable on a host without a GPU.  Pointers are made-up addresses that no accepted call is made with."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from memory_lean_optimizer_gb300 import build, lmopt
    build.build()
    return lmopt


P, U = 0x10000, 0x10001


def refused(lib, fn, code, *args):
    with pytest.raises(lib.LmoptError) as e:
        fn(*args)
    assert e.value.code == code, e.value


def test_cross_entropy_forward(lib):
    ok = dict(hidden=P, ldh=64, weight=P, ldw=64, target=P, rows=4, dim=64, vocab=10, ignore=-100, loss=P, lse=P, work=P,
              nbytes=1 << 40)
    call = lambda **kw: (lib.loss_xent_forward, kw.pop("code", lib.OPTIM_EINVAL), *{**ok, **kw}.values())
    for kw in (dict(rows=-1), dict(dim=0), dict(vocab=0), dict(rows=(1 << 28) + 1), dict(hidden=None), dict(weight=None),
               dict(target=None), dict(loss=None), dict(lse=None), dict(ldh=63), dict(ldw=63), dict(work=None), dict(nbytes=0),
               dict(hidden=U, code=lib.OPTIM_EALIGN), dict(weight=U, code=lib.OPTIM_EALIGN),
               dict(target=P + 4, code=lib.OPTIM_EALIGN), dict(lse=P + 2, code=lib.OPTIM_EALIGN),
               dict(work=P + 128, code=lib.OPTIM_EALIGN)):
        refused(lib, *call(**kw))


def test_cross_entropy_backward(lib):
    ok = dict(hidden=P, ldh=64, weight=P, ldw=64, target=P, lse=P, grad=P, rows=4, dim=64, vocab=10, ignore=-100, dh=P,
              lddh=64, dw=P, lddw=64, work=P, nbytes=1 << 40)
    call = lambda **kw: (lib.loss_xent_backward, kw.pop("code", lib.OPTIM_EINVAL), *{**ok, **kw}.values())
    for kw in (dict(grad=None), dict(lse=None), dict(lddh=1), dict(lddw=1), dict(nbytes=100),
               dict(dh=U, code=lib.OPTIM_EALIGN), dict(dw=U, code=lib.OPTIM_EALIGN), dict(grad=P + 1, code=lib.OPTIM_EALIGN)):
        refused(lib, *call(**kw))


def test_workspaces(lib):
    with pytest.raises(lib.LmoptError):
        lib.loss_xent_workspace(-1, 64, 10, P, 64, False)
    with pytest.raises(lib.LmoptError):
        lib.norm_layer_workspace(4, 0)
    f = lib.loss_xent_workspace(8192, 4096, 131072, P, 4096, False)
    b = lib.loss_xent_workspace(8192, 4096, 131072, P, 4096, True)
    logits = 8192 * 131072 * 2
    assert f < logits / 10 and b < logits / 2      # far below the logits, even in bf16
    # a weight that has to be copied on the way is copied by pieces
    assert lib.loss_xent_workspace(8192, 4096, 131072, P + 2, 4096, True) < b + (300 << 20)
    assert lib.norm_layer_workspace(0, 64) > 0
    n = ctypes.c_size_t()
    assert lib.load().loss_xent_workspace(4, 64, 10, P, 64, 1, None) == lib.OPTIM_EINVAL
    assert lib.load().loss_xent_workspace(4, 64, 10, P, 64, 1, ctypes.byref(n)) == lib.OPTIM_OK


def test_sizes_past_the_kernels_numbers(lib):
    for rows, dim, vocab in (((1 << 28) + 1, 8, 8), (1 << 26, 8, 1 << 26), (8, 1 << 26, 1 << 26), (1 << 27, 1 << 20, 8)):
        with pytest.raises(lib.LmoptError):
            lib.loss_xent_workspace(rows, dim, vocab, P, dim, True)
