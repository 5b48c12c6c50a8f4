"""The reader of lists of tensors behind clip_grad_norm, on host tensors (DLPack's device kind 1), against the
tensors' attributes."""
import ctypes
import timeit

import pytest
import torch

import fp4_precision_gemm_b200 as fq

CPU = 1
F, B = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    import os
    if not os.path.exists(fq.lists_path):
        from fp4_precision_gemm_b200 import build
        build.build()


def read(grads, outs=None, kind=CPU):
    items = (ctypes.c_int64 * max(4 * len(grads), 4))(*[-7] * max(4 * len(grads), 4))
    r = fq._lists()
    if r is None:
        pytest.skip("this torch has no DLPack exchange interface")
    return r(grads, outs, kind, ctypes.addressof(items)), list(items)


def test_items_are_the_attributes():
    base = torch.randn(1000)
    grads = [base, base[3:77], base.view(10, 100)[2:4], torch.zeros((3, 5), dtype=B), torch.zeros((0, 4)), torch.tensor(2.0),
             torch.nn.Parameter(torch.zeros(6, dtype=B)), torch.zeros((4, 4), requires_grad=True), torch.zeros((7, 1))[:, :1],
             torch.zeros((1, 9)).t(), base.bfloat16()[5:6], torch.empty((2, 0, 3), dtype=B)]
    assert all(g.is_contiguous() for g in grads)
    outs = [torch.empty_like(g.detach()) for g in grads]
    for o in (None, outs, grads):
        index, items = read(grads, o)
        assert index == 0
        want = [v for g, q in zip(grads, o or grads)
                for v in (g.data_ptr(), q.data_ptr(), g.numel(), fq.FP8Q_BF16 if g.dtype == B else fq.FP8Q_FP32)]
        assert items == want


class Other(torch.Tensor):
    pass


@pytest.mark.parametrize("bad", [torch.zeros(4, dtype=torch.float16), torch.zeros(4, dtype=torch.int32),
                                 torch.zeros(4, dtype=torch.float64), torch.zeros((4, 4)).t(), torch.zeros(8)[::2],
                                 torch.zeros((2, 1)).expand(2, 3), torch.zeros(4, dtype=torch.complex64), None, 3, [],
                                 torch.zeros(4).to_sparse(), torch.zeros(4).as_subclass(Other),
                                 torch.zeros(4, device="meta")], ids=lambda b: type(b).__name__)
def test_anything_else_is_left_to_the_attributes(bad):
    good = torch.zeros(4)
    assert read([good])[0] == 0
    assert read([good, bad])[0] == -1 and read([bad])[0] == -1
    assert read([good, good], [good, bad])[0] == -1
    assert read([good])[0] == 0                                    # and no error of the interpreter is left behind


def test_outputs_that_do_not_match():
    a, b = torch.zeros(4), torch.zeros(4, dtype=B)
    assert read([a, b], [torch.zeros(4), torch.zeros(4, dtype=B)])[0] == 0
    assert read([a], [torch.zeros(5)])[0] == -1 and read([a], [b])[0] == -1 and read([a, b], [a])[0] == -1
    assert read([a], (a,))[0] == -1                                # lists only
    assert read([a], kind=fq._DL_CUDA)[0] == -1                    # host tensors


def test_reading_hundreds_of_tensors():
    """The reader takes less than half the time of the attributes that it stands for (measured: a sixth)."""
    grads = [torch.zeros(100) for _ in range(300)]
    outs = [torch.zeros(100) for _ in range(300)]
    items = (ctypes.c_int64 * 1200)()
    r = fq._lists()
    if r is None:
        pytest.skip("this torch has no DLPack exchange interface")

    def attributes():
        for ts in (grads, outs):
            [t.data_ptr() for t in ts], [t.numel() for t in ts], [t.dtype for t in ts]
            [t.get_device() for t in ts], [t.is_contiguous() for t in ts]

    best = lambda f: min(timeit.repeat(f, number=20, repeat=7))  # noqa: E731
    assert best(lambda: r(grads, outs, CPU, ctypes.addressof(items))) < 0.5 * best(attributes)


def test_a_torch_without_the_interface():
    """No capsule, or one of another name: no table, and no error of the interpreter is left behind."""
    L = ctypes.PyDLL(fq.lists_path)
    L.fp8q_lists_api.argtypes, L.fp8q_lists_api.restype = [ctypes.py_object], ctypes.c_void_p
    new = ctypes.pythonapi.PyCapsule_New
    new.argtypes, new.restype = [ctypes.c_void_p, ctypes.c_char_p, ctypes.c_void_p], ctypes.py_object
    assert L.fp8q_lists_api(None) is None and L.fp8q_lists_api(new(0x1000, b"other", None)) is None
