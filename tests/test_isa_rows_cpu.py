"""Static checks on the gfx950 assembly of the row operators' kernels (no GPU
needed): no scratch, subnormals kept, no packed binary32 arithmetic, 16-byte
accesses, and the register and LDS budgets their launches count on."""
import importlib.util
import os
import re

import pytest

from tests.conftest import ROOT


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{mangled name: (body, metadata)} for every kernel."""
    spec = importlib.util.spec_from_file_location(
        "_ew_build", os.path.join(ROOT, "memory_bound_elementwise_amd", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    path = mod.device_asm(str(tmp_path_factory.mktemp("asm")), sources=mod.ROW_KERNEL_SOURCES)
    text = open(path).read()
    bodies = dict(re.findall(r"\n(_ZN2ew\w+):[^\n]*\n(; %bb\.0:.*?)\n\.Lfunc_end", text, re.S))
    meta = {k: dict(re.findall(r"\.amdhsa_(\w+) (\S+)", m)) for k, m in
            re.findall(r"\.amdhsa_kernel (\w+)(.*?)\.end_amdhsa_kernel", text, re.S)}
    assert bodies and set(bodies) == set(meta)
    return {k: (bodies[k], meta[k]) for k in bodies}


def test_every_kernel(kernels):
    assert len(kernels) > 60
    for name, (body, d) in kernels.items():
        assert d["private_segment_fixed_size"] == "0", name
        assert d["float_denorm_mode_32"] == "3" and d["float_denorm_mode_16_64"] == "3", name
        assert int(d["group_segment_fixed_size"]) <= 34 * 1024, name
        for pat in (r"\bv_pk_(add|mul|fma)_f32\b", r"\bv_cvt_pkrtz", r"\bscratch_"):
            assert not re.search(pat, body), (name, pat)


def test_no_atomics(kernels):
    """A call repeated gives the same bits."""
    for name, (body, _) in kernels.items():
        assert not re.search(r"\b(global|flat|buffer|ds)_\w*atomic|\bds_(add|or|max|min)_", body), name


def test_streams_use_16_byte_accesses(kernels):
    for name, (body, _) in kernels.items():
        if re.search(r"norm_row|norm_grad|vocab_forward|logprobs_grad|distill_grad", name):
            assert re.search(r"global_load_dwordx4 .* nt\b", body), name
        if re.search(r"norm_row_kernel\w*ELb0E|norm_grad_kernel|logprobs_grad|distill_grad", name):
            assert re.search(r"global_store_dwordx4 .* nt\b", body), name
        if re.search(r"logprobs_grad|distill_grad", name):      # rows on 16-byte boundaries
            assert re.search(r"buffer_store_dwordx4 .* nt sc1\b", body), name


def test_registers_of_16_bit_forward_kernels(kernels):
    """Eight waves a SIMD: at most 64 of its 512 registers a lane each."""
    names = [k for k in kernels if "vocab_forward" in k and "DF16" in k]
    assert len(names) == 2 * 5
    for name in names:
        assert int(kernels[name][1]["next_free_vgpr"]) <= 64, name


def test_registers_of_whole_row_kernels(kernels):
    """A row's block must fit a CU: 512 registers a lane and SIMD, shared by
    the block's waves on it."""
    for name, (_, d) in kernels.items():
        m = re.search(r"norm_row_kernelI\w*?Li(\d+)ELi\d+ELb", name)
        if m:
            assert int(d["next_free_vgpr"]) <= 512 // max(1, int(m.group(1)) // 4), name


def test_e4m3_conversion_is_the_hardware_one(kernels):
    for name, (body, _) in kernels.items():
        if re.search(r"norm_row_kernel\w*ELb1E", name):
            assert re.search(r"\bv_cvt_pk_fp8_f32\b", body), name
