"""The compiler resource report (CPU; hipcc only): readable names, and the named default kernels among those built."""
import os

from memory_bound_decode_gemv_amd import _build, profiling


def test_sixteen_bit_kernels_have_readable_names():
    names = ["_ZN2dg12_GLOBAL__N_113k_sample_pickIDF16bEEvPKT_PNS0_8RowSpaceENS0_10SampleArgsE",
             "_ZN2dg12_GLOBAL__N_113k_sample_pickIDF16_EEvPKT_PNS0_8RowSpaceENS0_10SampleArgsE",
             "_ZN2dg12_GLOBAL__N_113k_sample_pickIfEEvPKT_PNS0_8RowSpaceENS0_10SampleArgsE"]
    got = profiling._demangle(names)
    for name, kind in zip(got, ("__bf16", "_Float16", "float")):
        assert name.startswith(f"void dg::(anonymous namespace)::k_sample_pick<{kind}>({kind} const*, ")
        assert name.endswith("RowSpace*, dg::(anonymous namespace)::SampleArgs)")


def test_named_default_kernels_are_built():
    """The report names them by template and arguments, which have to be those of the sources."""
    sources = [os.path.join(_build.CSRC, n) for n in ("gemv_q4_0_mfma.hip", "gemv_qmfma_res.hip", "gemv_dense.hip")]
    built = {r["norm"] for r in profiling.kernel_records(sources)}
    asked = [k for _, k in profiling.DEFAULT_KERNELS if k.startswith(("k_qmfma<", "k_qres<", "k_gemv_"))]
    assert len(asked) == 5 and not [k for k in asked if k not in built]
