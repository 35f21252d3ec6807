"""Which kernel the grouped product with an epilogue runs (gmm_get_tile_config of
its operations), on the CPU: the rule counts 256 compute units there, as on the
MI355X.  The GPU tests of each kernel ask the same question first."""
import ctypes

import pytest

import moe_grouped_gemm_gmm_amd as gmm
import test_gpu_linear_forms as forms

NULL, SHAPE, DTYPE = 1, 2, 4
FWD, BWD = gmm.OP_BF16_LINEAR, gmm.OP_BF16_LINEAR_BWD


@pytest.mark.parametrize("name", list(forms.FORMS))
def test_forms_are_the_ones_meant(name):
    assert forms.chosen(name) == forms.FORMS[name][4:]


def test_every_kernel_of_the_rule_is_tested():
    got = {f[4:] for f in forms.FORMS.values()}
    assert {f[:1] for f in got} == {(1,), (2,), (3,)}
    assert {f for f in got if f[0] == 1} == {(1, 8, 16, 32), (1, 4, 16, 64), (1, 4, 32, 64)}
    assert {f for f in got if f[0] == 2} == {(2, 4, 128, 128), (2, 4, 128, 256)}
    assert {f[2] for f in got if f[0] == 3} >= {64, 96, 128, 160}


def test_the_choice_of_the_shapes_measured():
    def c(M, G, K, N, op=FWD):
        v = gmm.get_tile_config(op, M, K, N, G)
        return v["kernel"], v["tile_m"], v["tile_n"]
    assert c(8, 256, 512, 2048) == (1, 16, 64)
    assert c(1777, 13, 1088, 704) == (1, 32, 64)
    assert c(8192, 32, 2048, 512) == (3, 96, 256)
    assert c(65536, 256, 512, 2048) == (3, 160, 256)
    assert c(65536, 256, 2048, 512) == (3, 160, 256)
    assert c(8192, 32, 512, 2048) == (2, 128, 128)
    assert c(12000, 60, 1024, 1024) == (2, 128, 256)
    assert c(60000, 256, 64, 2048) == (2, 128, 128)
    assert c(8192, 32, 2048, 512, BWD)[0] == 3 and c(301, 5, 512, 192, BWD)[0] == 4


@pytest.mark.parametrize("op", [FWD, BWD])
def test_refusals(op):
    lib = gmm.load_library()
    cfg = gmm.TileConfig()
    get = lambda M=100, K=128, N=192, G=4, ot=1, p=cfg: lib.gmm_get_tile_config(op, M, K, N, G, 1, ot, ctypes.byref(p) if p else None)
    assert get() == 0
    assert get(p=None) == NULL and get(ot=2) == DTYPE
    assert get(M=0) == SHAPE and get(K=100) == SHAPE and get(N=32) == SHAPE and get(G=0) == SHAPE
    assert lib.gmm_set_tile_config(op, ctypes.byref(cfg)) == SHAPE       # no override
