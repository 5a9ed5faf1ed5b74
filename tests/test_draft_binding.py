"""CPU tests of the checks that the binding of the draft operators makes before a
call: the shapes of matrices."""
import pytest
import torch

from speculative_decoding_rejection_gb300 import draft as D

HOST = -1   # Tensor.get_device() of a host tensor
BF16 = torch.bfloat16


@pytest.mark.parametrize("shape", [(6, 8), (9, 8), (48,), (60,), (2, 3, 8), (6, 2, 4), (1, 6, 8), (6, 1, 8)])
def test_matrices_of_the_right_rows_pass(shape):
    """Rows of 8, at least 6 of them, however they are viewed; flat buffers too."""
    t = torch.zeros(shape, dtype=BF16)
    assert D._matrix("residual", t, BF16, 6, 8, HOST) == t.data_ptr()


@pytest.mark.parametrize("shape", [(8, 6), (4, 12), (2, 24), (16, 4, 5), (5, 8), (47,)])
def test_matrices_of_other_rows_are_refused(shape):
    with pytest.raises(ValueError):
        D._matrix("residual", torch.zeros(shape, dtype=BF16), BF16, 6, 8, HOST)


def test_no_matrix_and_other_types():
    assert D._matrix("residual", None, BF16, 6, 8, HOST) is None
    with pytest.raises(TypeError):
        D._matrix("residual", torch.zeros(6, 8), BF16, 6, 8, HOST)


@pytest.mark.gpu
def test_calls_refuse_transposed_matrices():
    import speculative_decoding_rejection_gb300 as sv

    def z(*shape, dtype=BF16):
        return torch.zeros(shape, dtype=dtype, device="cuda:0")

    M, N, K = 6, 8, 16
    x, w, y = z(M, K), z(N, K), z(M, N)
    for kw in (dict(residual=z(N, M)), dict(out=(z(N, M), None)), dict(out=(y, z(N, M)))):
        with pytest.raises(ValueError):
            sv.spec_head_forward(x, w, **kw)
    ok = (z(M, K), z(N, K), z(N, dtype=torch.float32))
    for kw in (dict(pre=z(N, M)), dict(out=(z(K, M), *ok[1:])), dict(out=(ok[0], z(K, N), ok[2]))):
        with pytest.raises(ValueError):
            sv.spec_head_backward(y, x, w, **{"pre": y, **kw}, act=sv.SPEC_ACT_SILU)
    cu = torch.tensor([0, M], dtype=torch.int32, device="cuda:0")
    with pytest.raises(ValueError):
        sv.spec_process_logits(y, cu, max_rows=M, out=z(N, M))
    with pytest.raises(ValueError):
        sv.spec_distill_loss(z(M + 1, N), y, cu, out=(z(M, dtype=torch.float32), z(N, M)))


class FakeDevice:
    entered = []

    def __init__(self, index):
        self.index = index

    def __enter__(self):
        self.entered.append(self.index)

    def __exit__(self, *_):
        self.entered.append(None)


@pytest.mark.parametrize("current,entered", [(0, [1, None]), (1, [])])
def test_a_call_runs_on_the_device_of_its_tensors(monkeypatch, current, entered):
    monkeypatch.setattr(FakeDevice, "entered", [])
    monkeypatch.setattr(torch.cuda, "device", FakeDevice)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    monkeypatch.setattr(D, "_current_device", lambda: current, raising=False)
    monkeypatch.setattr(D, "_raw_stream", lambda dev: 100 + dev)
    with D._Call(1, None, ()) as call:
        assert call.raw == 101 and FakeDevice.entered == entered[:1]
    assert FakeDevice.entered == entered


def test_a_stream_of_another_device_is_refused():
    class FakeStream:
        device = torch.device("cuda", 0)
        cuda_stream = 5

    with pytest.raises(ValueError):
        D._Call(1, FakeStream(), ())


def weights():
    p = [torch.zeros(4, requires_grad=True) for _ in range(3)]
    p[0].grad, p[1].grad = torch.ones(4), torch.ones(4)
    return p, [p[0].grad, p[1].grad.detach(), torch.ones(4)]   # the last one is not autograd's


def test_an_adamw_table_follows_the_gradients_of_its_weights():
    p, g = weights()
    table = D.SpecAdamwTable(None, 1, 32, (p, g, [], []))
    table.check()
    p[0].grad.add_(1)
    p[2].grad = torch.zeros(4)   # was none of the table's
    table.check()


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("new", [None, torch.zeros(4)])
def test_an_adamw_table_refuses_gradients_that_moved(which, new):
    """zero_grad() leaves None, the next backward pass another tensor."""
    p, g = weights()
    table = D.SpecAdamwTable(None, 1, 32, (p, g, [], []))
    p[which].grad = new
    with pytest.raises(ValueError, match="gradient"):
        table.check()


@pytest.mark.gpu
def test_an_adamw_step_refuses_gradients_that_moved():
    import speculative_decoding_rejection_gb300 as sv
    p = torch.ones(300, device="cuda:0", requires_grad=True)
    (p * p).sum().backward()
    state = [[torch.zeros(300, device="cuda:0")] for _ in range(2)]
    table = sv.spec_adamw_table([p], [p.grad], *state)
    for step in (1, 2):
        p.grad.zero_()
        (p * p).sum().backward()
        assert sv.spec_get_status(sv.spec_adamw_step(table, step, lr=0.1)) == sv.SPEC_OK
    keep = p.detach().clone()
    p.grad = None
    (p * p).sum().backward()
    with pytest.raises(ValueError, match="gradient"):
        sv.spec_adamw_step(table, 3, lr=0.1)
    assert torch.equal(p, keep)
