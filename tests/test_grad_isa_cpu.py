"""Checks on the gfx950 assembly of the gradient operators' kernels (host only).

No packed FP32 operations, no scalar-cache writes, no flat memory accesses (a pointer
whose address space was lost would be read by them), LDS within a compute unit's, and
the instructions the designs rest on.
"""
import importlib.util
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = ("act_kernels.hip", "wgrad_kernels.hip", "embed_kernels.hip", "policy_kernels.hip")


@pytest.fixture(scope="module")
def assembly():
    spec = importlib.util.spec_from_file_location(
        "_zs_build_grad", os.path.join(ROOT, "zero_sharded_mixed_shard_amd", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert set(SOURCES) <= set(mod.KERNEL_SOURCES)
    return {src: mod.device_assembly(src) for src in SOURCES}


def count(text, op):
    return len(re.findall(r"\b" + re.escape(op), text))


@pytest.mark.parametrize("src", SOURCES)
def test_forbidden_instructions(assembly, src):
    text = assembly[src]
    for op in ("v_pk_fma_f32", "v_pk_mul_f32", "v_pk_add_f32", "v_cvt_pkrtz_f16_f32",
               "flat_load", "flat_store", "flat_atomic", "global_atomic_add_f32",
               "global_atomic_pk_add"):
        assert count(text, op) == 0, op
    assert not re.search(r"\bs_(store|atomic|buffer_store|buffer_atomic|scratch_store)\w*", text)
    assert not re.search(r"\bs_dcache_(wb|discard)\w*", text)


@pytest.mark.parametrize("src", SOURCES)
def test_lds_fits_a_compute_unit(assembly, src):
    sizes = [int(x) for x in re.findall(r"\.amdhsa_group_segment_fixed_size (\d+)",
                                        assembly[src])]
    assert sizes and max(sizes) <= 160 * 1024


def test_the_designs_instructions(assembly):
    w = assembly["wgrad_kernels.hip"]
    assert count(w, "v_mfma_f32_32x32x16_bf16") > 0 and count(w, "v_mfma_f32_32x32x16_f16") > 0
    assert count(w, "ds_read_b64_tr_b16") > 0
    assert count(w, "v_cvt_scalef32_pk_bf16_fp8") > 0 and count(w, "v_cvt_scalef32_pk_f16_fp8") > 0
    assert count(assembly["act_kernels.hip"], "v_cvt_pk_fp8_f32") > 0
    p = assembly["policy_kernels.hip"]
    assert count(p, "v_pk_max_i16") > 0 and count(p, "v_pk_min_u16") > 0


def test_two_rows_of_the_longest_loss_share_a_compute_unit(assembly):
    # 512 lanes x 9 LDS vectors of 16 B, twice, within 160 KB
    text = assembly["policy_kernels.hip"]
    m = re.search(r"\.amdhsa_kernel (\S*policy_row_kernelILi1ELi512ELi23ELi9E\S*)(.*?)"
                  r"\.end_amdhsa_kernel", text, re.S)
    size = int(re.search(r"\.amdhsa_group_segment_fixed_size (\d+)", m.group(2)).group(1))
    assert 2 * size <= 160 * 1024
