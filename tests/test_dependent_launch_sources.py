"""What the sources of the kernels under programmatic dependent launch have to keep to, and no run shows:
such a kernel may be resident while the one before it still writes what it will read."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "semi_structured_sparsity_step_b200",
                    "csrc")


def _code(name):
    """The source without its comments."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["block_norm.cu", "block_norm.cuh", "block_norm_bwd.cu", "block_norm_bwd.cuh",
                                  "gemm_w8a8.cu", "grad_group.cu"])
def test_nothing_is_read_as_constant_for_the_kernel_s_life(name):
    """A read-only load (__ldg, ld.global.nc) asks for memory that nobody writes while the kernel runs, and a
    __restrict__ pointer lets the compiler choose one, or move the load ahead of the wait."""
    assert re.findall(r"__ldg\s*\(|\.nc\b|__restrict__", _code(name)) == []


def test_scales_of_the_tensor_core_products_are_no_read_only_loads():
    assert re.findall(r"__ldg\s*\([^;]*\b(?:amax|wmax|gamma)\b", _code("gemm_tc.cu")) == []


def test_the_8_bit_product_releases_its_successor_behind_its_own_wait():
    """The decode products read packed weights ahead of their wait, which holds only where every kernel before
    them had waited when it released them: the full-batch form of the 8-bit product too."""
    code = _code("gemm_tc.cu")
    body = code[code.index("tc_gemm_pair_kernel("):]
    wait = body.index("pdl_wait();")
    before, after = body[:wait], body[wait:]
    assert before.count("pdl_launch_dependents()") == \
        len(re.findall(r"if constexpr \(!epi_w8\(EPI\)\) \{\s*if \([^;{}]*\) pdl_launch_dependents\(\);\s*\}", before))
    assert re.match(r"pdl_wait\(\);\s*if constexpr \(epi_w8\(EPI\)\) \{\s*if \([^;{}]*\) pdl_launch_dependents\(\);\s*\}",
                    after)


@pytest.mark.parametrize("name", ["gemv_direct.cu", "gemv_tma.cu", "pack_gemv.cu"])
def test_activations_of_the_decode_products_are_no_read_only_loads(name):
    """Codes that the block norm writes while the product behind it is already there."""
    loads = re.findall(r"__ldg\s*\([^;]*", _code(name))
    assert [x for x in loads if re.search(r"\bxr\b|\bp \+ q\b", x)] == []
