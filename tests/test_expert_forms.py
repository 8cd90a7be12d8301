"""The cases of test_gpu_expert_forms.py take the kernel forms they are meant
for, by the library's own rules (CPU): a change of those rules that would leave
a kernel without its tests fails here."""
import pytest

import expert_cases as cases
import forms


def test_f8_cases_take_their_forms():
    assert set(cases.F8) == {"rows1", "rows2", "rows3", "rows4"} | set(forms.TILES)
    for form, shapes in cases.F8.items():
        for M, N, K in shapes:
            assert forms.f8(M, N) == form, (form, M, N)
            assert K % 128, (form, K)                  # a short last block
    odd = lambda K: -(-K // 128) % 2
    for form in ("quarter", "half"):                   # two blocks a step
        assert {odd(K) for _, _, K in cases.F8[form]} == {0, 1}, form
    for form in forms.TILES:                           # both ways to store y
        assert {N % 8 == 0 for _, N, _ in cases.F8[form]} == {True, False}, form


def test_f8_grouped_cases_take_their_forms():
    assert set(cases.F8_GROUPED) == {"rows1", "rows2", "rows4"} | set(forms.TILES)
    for form, groups in cases.F8_GROUPED.items():
        for counts, N, K, share, extra in groups:
            assert forms.f8_grouped(len(counts), sum(counts) + extra, N) == form, (form, counts, N)


@pytest.mark.parametrize("fmt", ["q4", "q8"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_block_quantized_cases_take_their_forms(fmt, act):
    for counts, N, K, share, extra in cases.TILES:
        assert forms.grouped(len(counts), sum(counts) + extra, N, K, fmt, act) == "tiles", (counts, N)
    assert {K // 64 % 4 for _, _, K, _, _ in cases.TILES} >= {0, 1, 2}
    for T, E, k, N, K in cases.TILE_LAYERS:
        assert forms.grouped(E, T * k, N, K, fmt, act) == "tiles"
    for form, groups in cases.FEW[fmt].items():
        for counts, N, K, share, extra in groups:
            assert forms.grouped(len(counts), sum(counts) + extra, N, K, fmt, act) == form, (form, counts, N)
