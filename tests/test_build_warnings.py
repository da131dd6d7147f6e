"""The build takes a compiler's warning for an error, above all that a loop was
not unrolled where the source asks for it: kernels then run with less in
flight than their comments say."""
import pytest

from lossless_bf16_exponent_zc_amd import build

NOT_UNROLLED = r"""
#include <hip/hip_runtime.h>
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
__global__ void k(const i32x8* a, f32x4* out, unsigned n) {
    f32x4 acc = {0, 0, 0, 0};
#pragma unroll 8
    for (unsigned b = threadIdx.x >> 6; b < n; b += 4)
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[b * 64], a[b * 64 + 1], acc, 0, 0, 0, 127, 0, 127);
    out[threadIdx.x] = acc;
}
"""
UNUSED = "int f(int x) { int y = x; return x; }"


@pytest.mark.parametrize("source,said", [(NOT_UNROLLED, "not unrolled"), (UNUSED, "unused variable")],
                         ids=["unroll", "unused"])
def test_a_warning_fails_the_build(tmp_path, monkeypatch, source, said):
    (tmp_path / "k.hip").write_text(source)
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    with pytest.raises(RuntimeError, match=said):
        build._compile("k.hip", [])
