"""What the experts' and gradient-norm calls refuse or promise beyond single arguments, on the CPU."""
import ctypes
import os
import re

import pytest

import matrix_orthogonalising_optimizer_muon_gb300 as mu
from matrix_orthogonalising_optimizer_muon_gb300 import experts

torch = pytest.importorskip("torch")
CSRC = os.path.join(os.path.dirname(os.path.abspath(mu.__file__)), "csrc")


class OnDevice:
    """Stands for a dense tensor of device 0, which this machine need not have."""
    is_cuda, device = True, "cuda:0"
    count = 0

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, torch.Size(shape)
        OnDevice.count += 1
        self.at = OnDevice.count << 32

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self, i):
        return self.shape[i + 1:].numel()

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


class Stream:
    cuda_stream = 0


def test_gradient_of_the_weights_needs_the_rows(monkeypatch):
    """dweights without rows: the call reaches the library with the rows' number above zero, so that it is refused, and
    never as one of no rows, which gives zeros.  What is not refused is not called here."""
    calls, lib = [], mu.load()

    class Library:
        @staticmethod
        def muon_expert_combine_backward(*args):
            calls.append(args)
            rows, expert_rows = args[8], args[4]
            return lib.muon_expert_combine_backward(*args) if rows > 0 and expert_rows is None else mu.MUON_OK
    monkeypatch.setattr(experts, "load", lambda: Library)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    f32, i32 = torch.float32, torch.int32
    dout, slots, w, dw = OnDevice(f32, 8, 40), OnDevice(i32, 8, 2), OnDevice(f32, 8, 2), OnDevice(f32, 8, 2)
    for drows in (None, OnDevice(f32, 16, 40)):
        with pytest.raises(mu.MuonError) as refused:
            mu.expert_combine_backward(dout, slots, w, drows=drows, dweights=dw, stream=Stream)
        assert refused.value.code == mu.MUON_ERR_INVALID_ARG
    # rows of a batch whose tokens chose nothing: an empty tensor says so
    mu.expert_combine_backward(dout, slots, w, rows=OnDevice(f32, 0, 40), dweights=dw, stream=Stream)
    assert [c[8] for c in calls] == [16, 16, 0]


@pytest.mark.parametrize("source,load", [("product.cu", "a.load("), ("wgrad.cu", "part_load<WIDE>(")])
def test_lanes_that_read_other_parts_are_ordered_behind_their_arrival(source, load):
    """One lane counts the parts of a cut tile and tells the others by a shuffle, which orders no memory: a warp barrier
    stands between the branch that the count decides and the first read of another CTA's part."""
    src = open(os.path.join(CSRC, source)).read()
    joins = re.findall(r"__shfl_sync\(0xffffffffu, seen, 0\) == (?:L\.)?parts - 1\) \{(.*?)" + re.escape(load), src, re.S)
    assert len(joins) == 1
    code = re.sub(r"//.*", "", joins[0])
    assert "__syncwarp();" in code


A, B = 0x100000000, 0x200000000   # far apart, 16-byte aligned, never dereferenced


@pytest.mark.parametrize("spec,norm", [
    ([(A, 100, 0)], A), ([(A, 100, 0)], A + 396), ([(A, 100, 0)], A + 200), ([(A, 101, 1)], A + 200),
    ([(A + 2, 1, 1)], A), ([(B, 7, 1), (A, 0, 0), (A, 100, 0)], A + 4), ([(B + k * 4096, 8, 0) for k in range(3000)], B + 2999 * 4096)])
def test_norm_does_not_lie_in_a_gradient(spec, norm):
    """A norm that would overwrite a value of the gradients: the first, the last, half of a pair of bf16 values."""
    n = len(spec)
    p, c, d = ((t * n)(*[x[i] for x in spec]) for i, t in enumerate((ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32)))
    # of a plan of no device, not read before the check
    handle = ctypes.cast(ctypes.create_string_buffer(b"\xff" * 256, 256), ctypes.c_void_p)
    assert mu.load().muon_grad_norm(handle, p, c, d, n, norm, None) == mu.MUON_ERR_INVALID_ARG


def test_the_room_for_copies_is_the_callers_choice():
    """A plan for the reductions, clipping and aligned products alone need not pay for copies of unaligned rows."""
    least, usual = mu.grad_plan_workspace_size(aligned_bytes=0), mu.grad_plan_workspace_size()
    assert least < 84e6 and usual - least < 230e6
    for more in (1, 256, 257, 1 << 34):
        assert mu.grad_plan_workspace_size(aligned_bytes=more) == least + (more + 255) // 256 * 256
    out, n = ctypes.c_void_p(), ctypes.c_int64()
    for bad in (-1, (1 << 34) + 1, -1 << 62):
        assert mu.load().muon_grad_plan_workspace_size_ex(bad, ctypes.byref(n)) == mu.MUON_ERR_INVALID_ARG
        assert mu.load().muon_grad_plan_create_ex(ctypes.byref(out), bad) == mu.MUON_ERR_INVALID_ARG and not out.value
    assert mu.load().muon_grad_plan_workspace_size_ex(0, None) == mu.MUON_ERR_INVALID_ARG
    assert mu.load().muon_grad_plan_create_ex(None, 0) == mu.MUON_ERR_INVALID_ARG


def test_clusters_beyond_the_portable_size_are_asked_for_first():
    """Eight CTAs always fit a cluster; whether sixteen do is the device's to say (one that is divided may lack a group of
    as many SMs), and a launch of a cluster that does not fit fails."""
    src = re.sub(r"//.*", "", open(os.path.join(CSRC, "experts.cu")).read())
    launch = src[src.index("cudaError_t launch_expert_order"):]
    launch = launch[:launch.index("\n}")]
    assert "cudaOccupancyMaxActiveClusters" in src and "places_sixteen() ? 4 : 3" in launch
