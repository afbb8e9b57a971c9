"""What the binding of the microscaled operators passes to the library, with a
recorder in the library's place: needs no GPU."""

from types import SimpleNamespace

import pytest
import torch

import quantized_weight_backward_amd as q
from quantized_weight_backward_amd import mx


class Recorder:
    """Stands for the library: keeps each call's name and arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0

        return call


@pytest.fixture
def recorder(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(mx, "lib", r)
    monkeypatch.setattr(mx, "_device_tensor", lambda t, name: t)
    monkeypatch.setattr(mx, "_elsewhere", lambda t, stream: False)
    monkeypatch.setattr(mx, "_handle", lambda: None)
    return r


def planes(rows, K):
    steps = -(-K // 256)
    return torch.zeros((rows, steps * 128), dtype=torch.uint8), torch.zeros((steps, rows, 8), dtype=torch.uint8)


def test_the_addresses_are_those_of_the_tensors_at_the_call(recorder):
    codes, scales = planes(5, 300)
    m = q.MXMatrix(codes, scales, 300)
    q.mx_mul_mat(m, m)
    old = codes.data_ptr(), scales.data_ptr()
    assert recorder.calls[-1][1][2:6] == old * 2
    kept = codes.data, scales.data  # the old storage stays taken, so the new lies elsewhere
    codes.data, scales.data = planes(5, 300)
    new = codes.data_ptr(), scales.data_ptr()
    assert not set(new) & set(old) and kept
    q.mx_mul_mat(m, m)
    assert recorder.calls[-1][1][2:6] == new * 2
    q.mx_dequantize(m)
    assert recorder.calls[-1][1][1:3] == new


def test_arrays_that_no_longer_fit_are_refused(recorder):
    def changed(change):
        codes, scales = planes(5, 300)
        m = q.MXMatrix(codes, scales, 300)
        change(codes, scales)
        made = len(recorder.calls)
        with pytest.raises(ValueError):
            q.mx_dequantize(m)
        with pytest.raises(ValueError):
            q.mx_mul_mat(m, m)
        assert len(recorder.calls) == made

    changed(lambda c, s: c.resize_(4, 256))
    changed(lambda c, s: c.resize_(5, 128))
    changed(lambda c, s: s.resize_(2, 4, 8))
    changed(lambda c, s: (c.resize_(6, 256), s.resize_(2, 6, 8)))
    changed(lambda c, s: setattr(c, "data", torch.zeros(5, 256)))


def test_a_view_of_a_made_matrix_is_the_caller_s_own(recorder):
    """Other storage for it is not the matrix's, neither in a call nor in its views."""
    m = q.mx_from_blocks(torch.zeros(5 * q.row_bytes(q.MXFP4, 320), dtype=torch.uint8), 320, 5)
    at = m.codes.data_ptr(), m.scales.data_ptr()
    c, s = m.codes, m.scales
    c.data, s.data = planes(5, 320)
    q.mx_dequantize(m)
    assert recorder.calls[-1][1][1:3] == at == (m.codes.data_ptr(), m.scales.data_ptr())


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Under such a stream the call would go back to the operands' device and
    run on that device's current stream instead."""
    monkeypatch.setattr(mx, "_device_tensor", lambda t, name: t)
    W = torch.zeros(5 * q.row_bytes(q.MXFP4, 320), dtype=torch.uint8)
    with pytest.raises(ValueError, match="stream"):
        q.mx_from_blocks(W, 320, 5, stream=SimpleNamespace(device=torch.device("cuda", 1)))


def test_a_result_of_another_type_is_refused(recorder):
    m = q.MXMatrix(*planes(5, 300), 300)
    for call in (lambda: q.mx_mul_mat_choice(300, 5, 5, torch.float64), lambda: q.mx_mul_mat(m, m, torch.float64),
                 lambda: q.mx_dequantize(m, torch.int32)):
        with pytest.raises(ValueError, match="dtype"):
            call()
