"""Checks on the gfx950 assembly of the kernels around a block's linear layers (host only).

No packed FP32 operations, no scalar-cache writes, no flat memory accesses, no atomics, LDS
within a compute unit's, and the instructions the designs rest on.
"""
import importlib.util
import os
import re
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = ("quant_kernels.hip", "product_kernels.hip", "dropout_kernels.hip",
           "residual_kernels.hip")


@pytest.fixture(scope="module")
def assembly():
    spec = importlib.util.spec_from_file_location(
        "_zs_build_block", os.path.join(ROOT, "zero_sharded_mixed_shard_amd", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert set(SOURCES) <= set(mod.KERNEL_SOURCES)
    with ThreadPoolExecutor(len(SOURCES)) as pool:
        return dict(zip(SOURCES, pool.map(mod.device_assembly, SOURCES)))


def count(text, op):
    return len(re.findall(r"\b" + re.escape(op), text))


def kernel(text, name):
    """The body of the first kernel whose symbol holds `name`."""
    sym = re.search(r"^(\S*" + name + r"\S*):", text, re.M)
    return text[sym.start():text.index("s_endpgm", sym.start())]


@pytest.mark.parametrize("src", SOURCES)
def test_forbidden_instructions(assembly, src):
    text = assembly[src]
    for op in ("v_pk_fma_f32", "v_pk_mul_f32", "v_pk_add_f32", "v_cvt_pkrtz_f16_f32", "flat_load",
               "flat_store", "flat_atomic", "global_atomic", "ds_add_f32"):
        assert count(text, op) == 0, op
    assert not re.search(r"\bs_(store|atomic|buffer_store|buffer_atomic|scratch_store)\w*", text)
    assert not re.search(r"\bs_dcache_(wb|discard)\w*", text)


@pytest.mark.parametrize("src", SOURCES)
def test_lds_fits_a_compute_unit(assembly, src):
    sizes = [int(x) for x in re.findall(r"\.amdhsa_group_segment_fixed_size (\d+)",
                                        assembly[src])]
    assert sizes and max(sizes) <= 160 * 1024


def test_the_products_instructions(assembly):
    p = assembly["product_kernels.hip"]
    assert count(p, "v_mfma_scale_f32_32x32x64_f8f6f4") > 0
    assert count(p, "v_mfma_f32_32x32x16_bf16") > 0
    assert count(p, "v_cvt_scalef32_pk_bf16_fp8") > 0
    # the large tile of 16-bit results: its steps' block holds all its products, the next
    # step's fragments and staging, and nothing that waits for spilled registers
    body = kernel(p, "product_tile_kernelILi1ELb1ELb0ELb0ELb0ELi256")
    blocks = re.split(r"^\.LBB", body, flags=re.M)
    steps = [b for b in blocks if "v_mfma" in b]
    assert len(steps) == 1
    assert count(steps[0], "v_mfma_scale_f32_32x32x64_f8f6f4") == 32
    assert count(steps[0], "ds_read_b128") == 32 and count(steps[0], "ds_write_b128") == 16
    assert count(steps[0], "global_load_dwordx4") == 16
    assert "scratch_" not in steps[0] and "v_accvgpr" not in steps[0]


def test_sixteen_bit_results_take_the_8_bit_instruction_and_fp32_the_bf16_one(assembly):
    p = assembly["product_kernels.hip"]
    for tile in (64, 128, 256):
        k = kernel(p, f"product_tile_kernelILi2ELb0ELb0ELb0ELb0ELi{tile}")
        assert "f8f6f4" not in k and "v_mfma_f32_32x32x16_bf16" in k
        k = kernel(p, f"product_tile_kernelILi0ELb1ELb0ELb0ELb0ELi{tile}")
        assert "f8f6f4" in k and "x16_bf16" not in k


def test_square_blocks_are_transposed_by_byte_permutes(assembly):
    q = assembly["quant_kernels.hip"]
    assert count(kernel(q, "quant_square_kernelILi1ELb1ELb0E"), "v_perm_b32") >= 32
    assert count(q, "v_cvt_pk_fp8_f32") > 0


def test_the_masks_multiplications_are_wide(assembly):
    d = assembly["dropout_kernels.hip"]
    # a block of four words: 20 products of 32 x 32 bits, high and low word each at once
    assert count(d, "v_mad_u64_u32") >= 20
