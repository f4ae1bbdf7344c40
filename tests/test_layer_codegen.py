"""Checks of the gfx950 code the recurrent layer's kernels compile to (CPU only:
hipcc cross-compiles): no instruction reads a register that the register
allocator left undefined, no kernel uses scratch memory, and none has packed
FP32 instructions."""
import pytest

import test_ssm_codegen as other

FILES = ("vdc_recurrence.hip", "vdc_layer_norm.hip", "vdc_pool.hip")


@pytest.mark.parametrize("name", FILES)
def test_scratch_and_instructions(name, tmp_path):
    other.test_scratch_and_instructions(name, tmp_path)


@pytest.mark.parametrize("name", FILES)
def test_no_read_of_undefined_registers(name):
    other.test_no_read_of_undefined_registers(name)
