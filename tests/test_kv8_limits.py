"""What the 8-bit cache's calls refuse before anything is launched: arrays that overlap in the
plan, misaligned arrays, overlapping output rows (no GPU)."""
import ctypes

import pytest

from tests.test_kv8 import P, expect, lib  # noqa: F401  (the fixture)

#       B max_pages max_rows capacity, then kv_len new_len held free n_free | table row_start kv_out held_out slots positions row_seq status
PLAN = [4, 8, 32, 10] + [ctypes.c_void_p(4096 * (i + 1)) for i in range(13)] + [None]
INPUTS, OUTPUTS = range(4, 9), range(9, 17)


@pytest.mark.parametrize("out", OUTPUTS)
def test_plan_refuses_an_output_that_is_another_array(lib, out):  # noqa: F811
    for other in list(INPUTS) + [o for o in OUTPUTS if o != out]:
        a = list(PLAN)
        a[out] = a[other]
        expect(lib, lib.spec_kv8_plan(*a), "SPEC_E_INVAL", b"one of the inputs" if other in INPUTS else b"same")


def test_plan_refuses_misaligned_arrays(lib):  # noqa: F811
    for i in list(INPUTS) + list(OUTPUTS):
        for off in (1, 2) + ((4,) if i == 13 else ()):          # slots are 64-bit numbers
            a = list(PLAN)
            a[i] = ctypes.c_void_p(a[i].value + off)
            expect(lib, lib.spec_kv8_plan(*a), "SPEC_E_INVAL", b"aligned")


def test_append_and_attention_refuse_misaligned_arrays(lib):  # noqa: F811
    append = [9, 2, 128, 1, 4, 5, P, P, P, P, P, P, P, 1, 256, 256, None]
    n = lib.spec_kv8_attention_workspace_bytes(5, 8, 2, 128)
    attention = [9, 2, 128, 1, 4, 5, 8, P, P, P, P, P, P, 1024, 0.1, P, 1024, P, P, n, None]
    for call, good, arrays in ((lib.spec_kv8_append, append, (8, 9, 10)), (lib.spec_kv8_attention, attention, (9, 10, 11, 17))):
        for i in arrays:
            for off in (1, 2):
                a = list(good)
                a[i] = ctypes.c_void_p(4096 + off)
                expect(lib, call(*a), "SPEC_E_INVAL", b"aligned")


def test_attention_refuses_overlapping_output_rows(lib):  # noqa: F811
    n = lib.spec_kv8_attention_workspace_bytes(5, 8, 2, 128)
    for stride in (0, 8, 1016, -1016):
        a = [9, 2, 128, 1, 4, 5, 8, P, P, P, P, P, P, 1024, 0.1, P, stride, None, P, n, None]
        expect(lib, lib.spec_kv8_attention(*a), "SPEC_E_INVAL", b"overlap")
