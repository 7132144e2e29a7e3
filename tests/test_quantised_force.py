"""The test hook of the 8-bit product's tiles."""
import sparse_gemm_irregular_gb300 as sg


def test_force_refuses_what_the_rule_never_chooses():
    lib = sg.load()
    for args in ((48, 0), (256, 0), (72, 0), (-64, 0), (16, 1), (64, 2), (64, -1)):
        assert lib.spgemm_quantised_force(*args) == -1, args
    for args in ((64, 0), (240, 1), (144, 1), (0, 0)):
        assert lib.spgemm_quantised_force(*args) == 0
