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


def test_arrivals_on_another_cta_order_memory_beyond_their_own():
    """A release at CTA scope orders nothing for the CTA that waits: an arrival on a peer's barrier releases at
    cluster scope, or is relaxed where there is no memory to hand over."""
    import glob
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.abspath(mu.__file__)), "csrc")
    seen = []
    for path in glob.glob(os.path.join(csrc, "*.cu*")):
        for instr in re.findall(r"mbarrier\.arrive[.\w:]*", open(path).read()):
            if "shared::cluster" in instr:
                seen.append(instr)
    assert seen and all(".release.cluster." in i or ".relaxed.cluster." in i for i in seen), seen


def test_star_import_needs_no_torch():
    """The package's names, the layer side's among them, on a machine without torch, as before there was a layer side."""
    import os
    import subprocess
    import sys
    code = ("import sys; sys.modules['torch'] = None\n"
            "from matrix_orthogonalising_optimizer_muon_gb300 import *\n"
            "assert grad_plan_workspace_size() > 0 and callable(rmsnorm_forward) and Act8.__slots__")
    root = os.path.dirname(os.path.dirname(os.path.abspath(mu.__file__)))
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True)


def test_waits_for_another_cta_acquire_beyond_their_own():
    """The weight gradient's barriers that the pair's other CTA completes (operands, freed slots, accumulators):
    every wait on them acquires at cluster scope, as the pair GEMM's do."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.abspath(mu.__file__)), "csrc", "wgrad.cu")).read()
    waits = re.findall(r"mbar_((?:test_|try_)?wait\w*)\(\s*(?:e\.)?(\w+) \+ ([^;{]*?)\)\)", src)
    crossing = [(kind, bar, args) for kind, bar, args in waits if bar in ("ready", "empty", "tfull", "tempty")]
    assert {bar for _, bar, _ in crossing} == {"ready", "empty", "tfull", "tempty"}
    for kind, bar, args in crossing:
        assert kind.endswith("_cluster") or args.rstrip(" )").endswith("true"), (kind, bar, args)
    assert "mbar_test_wait(" not in src
