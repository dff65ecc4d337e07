"""The tensor-level calls of the layer operators read row strides from their
tensors: views whose rows overlap are refused, every other row stride reaches
the library as it is.  Host tensors stand in for device tensors and a recorder
for the library, so nothing is launched."""
import pytest

torch = pytest.importorskip("torch")

BF16 = torch.bfloat16


class OnGpu:
    """A host tensor that says it is on the GPU."""
    is_cuda = True

    def __init__(self, t):
        self._t = t

    def __getattr__(self, name):
        return getattr(self._t, name)


class Handle:
    R = 1


@pytest.fixture
def T(monkeypatch):
    import __graft_entry__

    __graft_entry__.build()
    from collective_datapath_atom_gb300 import torch_api

    torch_api.calls = calls = []
    for name in ("purlin_rms_norm", "purlin_rms_norm_backward", "purlin_grouped_matmul",
                 "purlin_grouped_matmul_weight_grad"):
        monkeypatch.setattr(torch_api, name,
                            lambda *a, _name=name, **kw: calls.append((_name, a, kw)))
    yield torch_api
    del torch_api.calls


def mat(*shape, dtype=BF16):
    return OnGpu(torch.zeros(*shape, dtype=dtype))


def expanded(*shape):
    """Every row the same storage: strides (..., 0, 1)."""
    return OnGpu(torch.zeros(shape[-1], dtype=BF16).expand(*shape))


def overlapping(rows, cols):
    return OnGpu(torch.zeros(rows * cols, dtype=BF16).as_strided((rows, cols), (cols - 8, 1)))


def norm(T, **kw):
    a = dict(x=mat(4, 64), weight=mat(64), handle=Handle(), residual=mat(4, 64), out=mat(4, 64),
             total=mat(4, 64))
    a.update(kw)
    return T.rms_norm(**a)


def backward(T, **kw):
    a = dict(dy=mat(4, 64), total=mat(4, 64), weight=mat(64), handle=Handle(), dtotal=mat(4, 64),
             dx=mat(4, 64), dweight=mat(64, dtype=torch.float32))
    a.update(kw)
    return T.rms_norm_backward(**a)


def groups():
    return dict(begin=mat(2, dtype=torch.int64), count=mat(2, dtype=torch.int64), handle=Handle())


def product(T, **kw):
    a = dict(x=mat(4, 64), w=mat(2, 32, 64), out=mat(4, 32), **groups())
    a.update(kw)
    return T.grouped_matmul(**a)


def grad(T, **kw):
    a = dict(dy=mat(4, 32), x=mat(4, 64), out=mat(2, 32, 64), **groups())
    a.update(kw)
    return T.grouped_matmul_weight_grad(**a)


def test_contiguous_operands_pass(T):
    for call in (norm, backward, product, grad):
        call(T)
    assert len(T.calls) == 4


@pytest.mark.parametrize("call,name,cols", [
    (norm, "x", 64), (norm, "residual", 64), (norm, "out", 64), (norm, "total", 64),
    (backward, "dy", 64), (backward, "total", 64), (backward, "dtotal", 64), (backward, "dx", 64),
    (product, "x", 64), (product, "out", 32), (grad, "dy", 32), (grad, "x", 64)])
@pytest.mark.parametrize("view", [expanded, overlapping])
def test_rows_that_overlap_are_refused(T, call, name, cols, view):
    """An expanded gradient, as autograd hands one over below a sum, has a row
    stride of 0, which the C call takes for contiguous rows: it would read or
    write rows * cols elements of a buffer of cols."""
    with pytest.raises(ValueError, match="overlap"):
        call(T, **{name: view(4, cols)})
    assert not T.calls


@pytest.mark.parametrize("call,name", [(product, "w"), (grad, "out")])
@pytest.mark.parametrize("count", [1, 2])
def test_stacks_whose_rows_overlap_are_refused(T, call, name, count):
    kw = {name: expanded(count, 32, 64)}
    if count == 1:
        kw.update(begin=mat(1, dtype=torch.int64), count=mat(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="overlap"):
        call(T, **kw)
    assert not T.calls


def test_pitched_rows_pass_with_their_stride(T):
    wide = OnGpu(torch.zeros(4, 80, dtype=BF16)[:, :64])
    norm(T, x=wide, total=wide)
    backward(T, dtotal=wide)
    product(T, x=wide)
    grad(T, x=wide)
    assert T.calls[0][2]["ldx"] == T.calls[0][2]["ldt"] == 80
    assert T.calls[1][2]["lddt"] == T.calls[2][2]["ldx"] == T.calls[3][2]["ldx"] == 80


@pytest.mark.parametrize("pitch", [1001, 1008, 1024])
def test_one_row_of_odd_length_passes(T, pitch):
    """Row strides have to be multiples of 16 bytes for the products; a single
    row has none."""
    x = OnGpu(torch.zeros(1, pitch, dtype=BF16)[:, :1001])
    one = dict(begin=mat(1, dtype=torch.int64), count=mat(1, dtype=torch.int64))
    product(T, x=x, w=OnGpu(torch.zeros(1, 32, 1008, dtype=BF16)[:, :, :1001]), out=mat(1, 32), **one)
    product(T, x=mat(1, 64), w=mat(1, 1, 64), out=mat(1, 1), **one)
    grad(T, dy=mat(1, 33), x=x, out=mat(1, 33, 1001), **one)
    grad(T, dy=mat(1, 1), x=x, out=OnGpu(torch.zeros(1, 1, pitch, dtype=BF16)[:, :, :1001]), **one)
    assert [c[2]["ldx"] for c in T.calls] == [1008, 64, 1008, 1008]
    assert T.calls[1][2]["ldw"] == 64 and T.calls[1][2]["ldy"] == 8
    assert T.calls[2][2]["lddy"] == 40 and T.calls[2][2]["lddw"] == 1001
    assert T.calls[3][2]["lddy"] == 8 and T.calls[3][2]["lddw"] == 1008


def test_matrices_of_one_row_lie_apart_as_their_stack_says(T):
    w = OnGpu(torch.zeros(2, 5, 64, dtype=BF16)[:, :1])
    product(T, w=w, out=mat(4, 1))
    assert T.calls[0][2]["ldw"] == 320


def test_one_row_in_place_keeps_one_stride(T):
    row = OnGpu(torch.zeros(1, 1008, dtype=BF16)[:, :1001])
    norm(T, x=row, weight=mat(1001), residual=row, out=row, total=None)
    kw = T.calls[0][2]
    assert kw["ldx"] == kw["ldr"] == kw["ldy"] == 1008


@pytest.mark.gpu
@pytest.mark.parametrize("pitch", [1001, 1008])
def test_one_odd_row_on_the_gpu(pitch):
    """Whole numbers: exact in any order.  The padding holds NaN."""
    import __graft_entry__

    __graft_entry__.build()
    from collective_datapath_atom_gb300 import torch_api as A

    def whole(*shape, cols):
        t = torch.full(shape, float("nan"), device="cuda", dtype=BF16)
        t[..., :cols] = torch.randint(-3, 4, (*shape[:-1], cols), device="cuda").bfloat16()
        return t[..., :cols]

    h = A.initialize(1, stream=torch.cuda.current_stream())
    try:
        k, n = 1001, 37
        x, dy = whole(1, pitch, cols=k), whole(1, 40, cols=n)
        w = whole(1, n, 1008, cols=k)
        begin = torch.zeros(1, device="cuda", dtype=torch.int64)
        count = torch.ones(1, device="cuda", dtype=torch.int64)
        y = A.grouped_matmul(x, w, begin, count, h)
        dx = A.grouped_matmul(dy, w, begin, count, h, transposed=True)
        dw = A.grouped_matmul_weight_grad(dy, x, begin, count, h)
        A.check(h)
        assert torch.equal(y, (x.double() @ w[0].double().t()).float().bfloat16())
        assert torch.equal(dx, (dy.double() @ w[0].double()).float().bfloat16())
        assert torch.equal(dw[0], (dy.double().t() @ x.double()).float().bfloat16())
        # rows of one element each, of a stack with a stride of its own
        w1 = whole(2, 3, 1008, cols=k)[:, :1]
        x2 = whole(2, 1008, cols=k)
        y = A.grouped_matmul(x2, w1, torch.arange(2, device="cuda"), torch.ones(2, device="cuda").long(), h)
        A.check(h)
        want = (x2.double() * w1[:, 0].double()).sum(1, keepdim=True)
        assert torch.equal(y, want.float().bfloat16())
    finally:
        A.finalize(h)
