"""Calls on several devices of one process, without a GPU: the library over a
stand-in for the HIP runtime (native/fake_devices.cpp) in a process of its own,
where each device has to be told of a kernel's large dynamic LDS."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")

START = """
import ctypes, sys, types

fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # in front of libmoe's own runtime
launches, refused, large = ((ctypes.c_int * 8).in_dll(fake, "fake_" + name)
                            for name in ("launches", "refused", "large"))
torch = sys.modules["torch"] = types.ModuleType("torch")  # would load the real runtime
torch.bfloat16 = torch.float32 = None
sys.path.insert(0, sys.argv[2])
from block_quantized_expert_amd import binding as B

lib, p = B.lib(), ctypes.c_void_p(0x10000)  # never dereferenced

def everywhere(what, call):
    # the same launches on every device, in any order
    counts = set()
    for device in (0, 3, 0, 1, 3):
        fake.fake_device(device)
        before = launches[device], large[device]
        assert call() == 0, (what, device)
        counts.add((launches[device] - before[0], large[device] - before[1]))
    assert len(counts) == 1, (what, counts)
    return counts.pop()[1]
"""

PRODUCTS = START + """
kind = sys.argv[3]
Weight = {"int8": B.MoeInt8Weight, "mxfp4": B.MoeMxfp4Weight}[kind]
forms = set()
for slots, rows in ((4096, 4096), (2048, 2048), (1024, 2048), (512, 4096), (333, 2048),
                    (256, 4096), (24, 4096), (1065, 7187), (647, 5641), (2309, 3357),
                    (33, 7465)):
    w = ctypes.byref(Weight(1, rows, 4096, 0x10000, 0x10000))
    tile = [ctypes.c_int32() for _ in range(3)]
    assert getattr(lib, "moe_%s_form" % kind)(1, rows, 4096, slots, 0, 0,
                                              *map(ctypes.byref, tile)) == 0
    for t in (0, 1):
        args = (p, p, slots, None, None, 0, p, t, rows, None)
        n = everywhere((slots, rows, t), lambda: getattr(lib, "moe_product_" + kind)(w, *args))
        everywhere((slots, rows, t), lambda: getattr(lib, "moe_swiglu_" + kind)(w, w, *args))
        assert n <= (tile[2].value > 0), (slots, rows)  # small tiles do without
        if n:
            forms.add((tile[0].value, tile[1].value))
assert len(forms) >= 3, forms
print("ok")
"""

LAYERS = START + """
def layer(kind, shared, packed=None, experts=16, hidden=4096, inter=2048):
    def proj(k):
        return B.MoeProj(k, 0x10000, 0x10000)
    g = proj(kind)
    s = proj(shared if shared is not None else kind)
    return B.MoeLayer(hidden, inter, experts, 4, g, g, g, int(shared is not None), inter, s, s, s,
                      packed)

X4, F8 = B.MOE_W_MXFP4, B.MOE_W_FP8E4M3_B128
seen = 0
for l in (layer(X4, None), layer(X4, X4), layer(X4, F8), layer(X4, X4, 0x10000),
          layer(X4, F8, 0x10000), layer(F8, None), layer(F8, F8), layer(F8, X4)):
    ref = ctypes.byref(l)
    for n in (1, 2, 8, 16, 40, 256, 1024):
        for x_type in (B.MOE_ACT_F32, B.MOE_ACT_BF16):
            for tau in (0.0, 0.5):
                opts = B.MoeOpts(lazy_tau=tau)
                seen += everywhere(
                    (l.gate.type, l.has_shared, bool(l.packed_experts), n, x_type, tau),
                    lambda: lib.moe_ffn_forward_ex(ref, p, x_type, n, p, p, p, p, p, p,
                                                   ctypes.byref(opts), p, 1 << 40, None, None,
                                                   None, None, None))
assert seen > 100, seen
print("ok")
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("fake") / "fake_devices.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__",
                    "-I" + os.path.join(ROCM, "include"), "-Wl,-soname,fake_devices.so",
                    os.path.join(ROOT, "tests", "native", "fake_devices.cpp"), "-o", out],
                   check=True)
    return out


def _run(*argv):
    r = subprocess.run([sys.executable, "-c", *argv], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


@pytest.mark.parametrize("kind", ["int8", "mxfp4"])
def test_products_run_on_every_device(fake, kind):
    _run(PRODUCTS, fake, ROOT, kind)


def test_layers_run_on_every_device(fake):
    _run(LAYERS, fake, ROOT)
