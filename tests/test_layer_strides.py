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
