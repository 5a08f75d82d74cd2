"""What the layer side refuses or promises beyond single arguments, on the CPU."""
import pytest

import matrix_orthogonalising_optimizer_muon_gb300 as mu

torch = pytest.importorskip("torch")


class OnDevice:
    """Stands for a uint8 tensor of a device, which this machine need not have."""
    dtype, is_cuda = torch.uint8, True

    def __init__(self, index, shape):
        self.device, self.shape = "cuda:%d" % index, shape
        self.index = index

    def dim(self):
        return 2

    def stride(self, i):
        return (self.shape[1], 1)[i]

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 1 << 32


def test_codes_and_scales_lie_on_one_device():
    mu.Act8(OnDevice(0, (4, 64)), OnDevice(0, (4, 16)), 50, "int8")
    with pytest.raises(ValueError, match="device"):
        mu.Act8(OnDevice(0, (4, 64)), OnDevice(1, (4, 16)), 50, "int8")
