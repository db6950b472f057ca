"""The Python calls around the step's attention refuse tables whose rows have another width than the parameters say:
the right number of elements, read with another width, would give other numbers.  No test here needs a GPU."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from test_step_host import Passed, bf16, f32, i32, lib, on_the_host, rotate_call, verify_call  # noqa: F401
from test_step_host import params

from paged_kv_gqa_02_gb300 import ops


@pytest.mark.parametrize("noise", [(2, 128), (4, 50), (1, 200), (1, 2, 128), (2, 2, 64), (1, 100), (3, 101)])
def test_noise_of_another_width(on_the_host, noise):
    with pytest.raises(ValueError, match="noise"):
        verify_call(noise=f32(*noise))


@pytest.mark.parametrize("noise", [(2, 100), (3, 100), (200,), (1, 2, 100)])
def test_noise_of_the_vocabularys_width(on_the_host, noise):
    with pytest.raises(Passed):
        verify_call(noise=f32(*noise))


@pytest.mark.parametrize("table", [(9, 128), (18, 32), (9, 65), (1, 576), (1, 9, 128)])
def test_cosines_and_sines_of_another_width(on_the_host, table):
    with pytest.raises(ValueError, match="table"):
        rotate_call(table=f32(*table))


@pytest.mark.parametrize("table", [(9, 64), (12, 64), (576,), (1, 9, 64)])
def test_cosines_and_sines_of_the_turning_dims_width(on_the_host, table):
    with pytest.raises(Passed):
        rotate_call(table=f32(*table))


def test_no_dims_turn_without_a_table(on_the_host):
    for table in (None, f32(0), f32(9, 64)):
        with pytest.raises(Passed):
            ops.rotate(params(), ops.make_rows(5, 3), ops.make_rope(0), bf16(5, 8, 64), bf16(5, 2, 64), i32(3), table, context_lens=i32(2),
                       q_out=bf16(5, 8, 64), k_out=bf16(5, 2, 64))


def test_a_store_without_all_of_the_cache_is_the_librarys_to_refuse(on_the_host):
    for missing in ("v_cache", "block_tables", "v"):
        with pytest.raises(Passed):
            rotate_call(**{missing: None})
