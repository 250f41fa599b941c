"""Static checks on the gfx950 assembly of the kernels of layer norm, the policy
loss and the movement of rows to experts (no GPU needed): 16-byte accesses,
registers and LDS that their launches count on.  (No scratch, no atomics, no
packed binary32 arithmetic and subnormals kept are checked for them too, with
every other row operator's kernels.)"""
import re

from tests.test_isa_rows_cpu import kernels  # noqa: F401  (the fixture)


def of(kernels, pattern):  # noqa: F811
    """{name: (body, metadata, match)} of the kernels whose name matches."""
    found = {k: (*v, m) for k, v in kernels.items() if (m := re.search(pattern, k))}
    assert found, pattern
    return found


def test_every_operator_has_its_kernels(kernels):  # noqa: F811
    for pattern, least in (("ew_layernorm_kernel", 3 * 20), ("ew_layernorm_back_kernel", 3 * 9),
                           ("ew_layernorm_long", 3), ("ew_layernorm_dx", 3), ("ew_policy_small", 6),
                           ("ew_policy_rows", 6), ("ew_policy_grad", 6), ("ew_experts_sort", 4),
                           ("ew_experts_gather", 9), ("ew_experts_combine_kernel", 21),
                           ("ew_experts_combine_grad", 18)):
        assert len(of(kernels, pattern)) >= least, pattern


def test_streams_use_16_byte_accesses(kernels):  # noqa: F811
    # rows shorter than a vector go by elements
    for name, (body, _, _) in of(kernels, r"layernorm_(kernelI\w+ELb0E|back_kernelI\w+ELb0E)").items():
        assert re.search(r"global_load_dwordx4 .* nt\b", body), name
        assert re.search(r"global_store_dwordx4 .* nt\b", body), name
    for name, (body, _, _) in of(kernels, r"layernorm_(long|dx)|experts_(gather|combine|combine_grad)_kernel"
                                          r"(?!\w*RowFitE2E)").items():
        assert re.search(r"global_load_dwordx4\b", body), name
        assert re.search(r"global_store_dwordx4\b", body), name
    # the rows of experts are read once, a token's own row stays for its choices
    for name, (body, _, _) in of(kernels, r"experts_combine_(grad_)?kernel(?!\w*RowFitE2E)").items():
        assert re.search(r"global_load_dwordx4 .* nt\b", body), name
    for name, (body, _, _) in of(kernels, r"policy_(small|rows|grad)_kernelILb[01]ELb0E").items():
        assert re.search(r"global_load_dwordx4 .* nt\b", body), name


def test_rows_in_registers_fit_a_cu(kernels):  # noqa: F811
    """512 registers a lane and SIMD, shared by a block's waves on it."""
    for name, (_, d, m) in of(kernels, r"layernorm_kernelI\w*?Li(\d+)ELi\d+ELi\d+ELb").items():
        waves = max(int(m.group(1)), 4)
        assert int(d["next_free_vgpr"]) <= 512 // (-(-waves // 4)), name
    for name, (_, d, m) in of(kernels, r"layernorm_back_kernelI\w*?Li(\d+)ELi\d+ELi(\d+)E").items():
        waves = int(m.group(1)) * int(m.group(2))
        assert int(d["next_free_vgpr"]) <= 512 // (-(-waves // 4)), name


def test_one_row_a_wave_leaves_room_for_eight(kernels):  # noqa: F811
    """Short rows' loads are hidden by other waves: eight a SIMD, 64 registers each."""
    for name, (_, d, _) in of(kernels, r"layernorm_kernelI\w+Li1ELi1ELi1ELb0E").items():
        assert int(d["next_free_vgpr"]) <= 64, name


def test_five_blocks_of_sequences_a_cu(kernels):  # noqa: F811
    """Their number is what the chip holds at once: five waves a SIMD."""
    for name, (_, d, _) in of(kernels, r"policy_(rows|parts)_kernel").items():
        assert int(d["next_free_vgpr"]) <= 96, name


def test_sums_of_a_batch_are_binary64(kernels):  # noqa: F811
    for name, (body, _, _) in of(kernels, r"policy_(small|rows|parts|join)_kernel").items():
        assert "v_add_f64" in body, name
    for name, (body, _, _) in of(kernels, r"layernorm_(long_)?kernel").items():
        assert re.search(r"v_(add|fma|fmac)_f64", body), name
