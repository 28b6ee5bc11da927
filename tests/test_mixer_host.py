"""Host side of the operators around the delta rule.  No GPU is needed."""
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import mixer_reference as R
import mixer_reference_flat as F
from gated_delta_rule_gdn_gb300 import _mixer, build

# A runtime whose calls succeed, but for the one named in FAIL; the current device is DEVICE.
RUNTIME = r'''
#include "residency.h"
#include <cstdio>
#include <cstdlib>
#include <cstring>
static const char* fail;
static int device, asked;
static cudaError_t answer(const char* name) { return fail && !strcmp(fail, name) ? cudaErrorInvalidValue : cudaSuccess; }
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = device; return answer("device"); }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) { a->sharedSizeBytes = 1024; return answer("attributes"); }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int v) { return v == 226 * 1024 ? answer("shared") : cudaErrorUnknown; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int d) { *v = 152; return d == device ? answer("sms") : cudaErrorUnknown; }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int, size_t) { ++asked; *n = 2; return answer("occupancy"); }
}
int main(int argc, char** argv) {
    device = atoi(argv[1]);
    fail = argc > 2 ? argv[2] : nullptr;
    static gdn::Residency r;
    int a = 0, b = 0;
    const cudaError_t e = r.get(&r, 192, 1000, &a), f = r.get(&r, 192, 1000, &b);
    printf("%d %d %d %d %d\n", (int)e, (int)f, a, b, asked);
}
'''


@pytest.fixture(scope="module")
def residency(tmp_path_factory):
    d = tmp_path_factory.mktemp("residency")
    (d / "main.cpp").write_text(RUNTIME)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc())))
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-I", os.path.join(cuda, "include"), "-I", build.CSRC,
                    "-I", build.INCLUDE, "-x", "c++", os.path.join(build.CSRC, "residency.cu"), str(d / "main.cpp"),
                    "-o", str(d / "run")], check=True)
    return lambda *args: [int(v) for v in subprocess.run([str(d / "run"), *map(str, args)], check=True, capture_output=True,
                                                         text=True).stdout.split()]


@pytest.mark.parametrize("device", [0, 63, 64, 1000])
def test_resident_blocks_of_any_device(residency, device):
    first, second, a, b, asked = residency(device)
    assert (first, second, a, b) == (0, 0, 304, 304)
    assert asked == (1 if device < 64 else 2)


@pytest.mark.parametrize("what", ["device", "attributes", "shared", "sms", "occupancy"])
@pytest.mark.parametrize("device", [0, 64])
def test_a_failed_query_is_an_error(residency, device, what):
    assert residency(device, what)[:2] == [1, 1]


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("cu", [None, [0, 0, 1, 3, 6, 6, 20, 22]])
@pytest.mark.parametrize("silu,given", [(True, True), (False, False)])
def test_flat_convolution_reference(W, cu, silu, given):
    """The whole-array reference against the one that goes token by token (sums of up to 22 terms in 64 bits)."""
    rng = np.random.default_rng(W)
    B, T, D = (1, 22, 3) if cu else (2, 11, 3)
    N = len(cu) - 1 if cu else B
    x, dy, w, b = rng.normal(size=(B, T, D)), rng.normal(size=(B, T, D)), rng.normal(size=(D, W)), rng.normal(size=D)
    h0, dhT = rng.normal(size=(2, N, W - 1, D)) if given else (None, None)
    got = F.conv(x, w, dy, b, silu, h0, dhT, cu)
    y, hT = R.conv_fwd(x, w, b, silu, h0, cu)
    want = dict(R.conv_bwd(x, w, dy, b, silu, h0, dhT, cu), y=y, hT=hT)
    mags = want.pop("abs")
    for name, v in want.items():
        assert np.allclose(got[name], v, rtol=1e-13, atol=1e-13), name
    for name, v in mags.items():
        assert np.allclose(got["abs"][name], v, rtol=1e-13), name


@pytest.mark.parametrize("change", ["torch", "python", "place", "gone"])
def test_another_torch_or_python_means_another_build(change, monkeypatch, tmp_path):
    """The extension module is of one torch and one Python: with another it is neither up to date nor loaded."""
    build.build()
    assert build.up_to_date() and build.native_current()
    version = open(os.path.join(build._torch_dir(), "version.py"), encoding="utf-8").read()
    if change in ("torch", "place"):
        (tmp_path / "version.py").write_text(version + ("git_version = 'another'\n" if change == "torch" else ""))
        monkeypatch.setattr(build, "_torch_dir", lambda: str(tmp_path))
    elif change == "python":
        monkeypatch.setattr(build.sys, "version", "3.99.0")
    else:
        monkeypatch.setattr(build, "STAMP", str(tmp_path / "no.stamp"))
    assert not build.native_current() and not build.up_to_date()
    monkeypatch.setattr(_mixer, "_NATIVE", None)
    with pytest.raises(RuntimeError, match="another torch or Python"):
        _mixer.native()
    monkeypatch.undo()
    assert build.up_to_date() and _mixer.native()


def _coefficients(function):
    """The decimal constants of one function of glr_math.cuh, as the fp32 numbers they become."""
    text = open(os.path.join(build.CSRC, "glr_math.cuh")).read()
    body = text[text.index(function):]
    return [float(np.float32(c)) for c in re.findall(r"-?\d+\.\d*(?:e[-+]?\d+)?(?=f\b)", body[:body.index("\n}")])]


def _stated(which):
    """The bound that a comment of glr_math.cuh gives behind these words."""
    text = open(os.path.join(build.CSRC, "glr_math.cuh")).read()
    return 2.0 ** -float(re.search(r"off by less than 2\^-([\d.]*\d)", text[text.index(which):]).group(1))


def test_polynomial_of_the_decay():
    """The bound that the comment states, for the coefficients in 64 bits; both forms have the same ones."""
    one, two = _coefficients("Decay decay(float& x) {"), _coefficients("void decay(float& x0, float& x1, Decay& d0, Decay& d1) {")
    assert one[3:10] == two[4:11] and one[9] == 0.5
    low, high = one[3], one[4]                            # ln 2 = -(high + low), high with zeros behind
    assert abs(-high - low - np.log(2)) < 2.0 ** -36 and (high * 2 ** 9).is_integer()
    r = np.linspace(-0.5 * np.log(2), 0.5 * np.log(2), 2_000_001)
    q = np.zeros_like(r)
    for c in one[5:10]:
        q = q * r + c
    assert np.abs(r + r * r * q - np.expm1(r)).max() < _stated("p = exp(r) - 1")


def test_polynomial_of_softplus():
    one, two = _coefficients("float softplus(float z, float q) {"), _coefficients("void softplus(float z0")
    q = np.linspace(2.0 ** -30, 1, 2_000_001)
    p = np.zeros_like(q)
    for c in one[:9]:
        p = p * q + c
    assert one[:9] == two[:9]
    assert np.abs(q * p / np.log1p(q) - 1).max() < _stated("log1p(q) = q P(q)")
