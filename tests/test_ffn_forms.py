"""Which kernel the gated block's calls run (gmm_get_tile_config of their
operations), on the CPU: the rule counts 256 compute units there, as on the
MI355X.  The GPU tests of each kernel ask the same question first."""
import ctypes

import pytest

import moe_grouped_gemm_gmm_amd as gmm
import test_gpu_ffn_forms as forms

NULL, SHAPE, DTYPE = 1, 2, 4
FWD, BWD, DW = gmm.OP_BF16_SWIGLU, gmm.OP_BF16_SWIGLU_BWD, gmm.OP_TGMM_MX8


def config(op, M, K, N, G):
    c = gmm.get_tile_config(op, M, K, N, G)
    assert c["depth"] == c["residency"] == c["placement"] == 0
    return c["kernel"], c["waves"], c["tile_m"], c["tile_n"]


@pytest.mark.parametrize("name", list(forms.FORMS))
def test_forms_are_the_ones_meant(name):
    assert forms.chosen(name) == forms.FORMS[name][4:]


def test_every_kernel_is_reached():
    assert config(FWD, 8, 2048, 512, 256) == (1, 8, 16, 32)             # one token of 256 experts
    assert config(FWD, 40, 192, 320, 2) == (1, 8, 32, 32)
    assert config(FWD, 203, 2048, 512, 16) == (1, 4, 16, 64)
    assert config(FWD, 200, 128, 320, 5) == (1, 8, 64, 32)
    assert config(FWD, 900, 448, 704, 4) == (2, 4, 128, 128)
    assert config(FWD, 3800, 128, 1344, 40) == (2, 4, 128, 256)
    assert config(FWD, 8192, 2048, 512, 32) == (3, 12, 160, 256)
    assert config(BWD, 301, 512, 192, 5) == (4, 4, 128, 128)
    assert config(BWD, 3100, 512, 512, 40) == (2, 4, 128, 128)          # dw's 256-column tiles keep the two apart
    assert config(BWD, 3800, 1344, 64, 40) == (2, 4, 128, 256)
    assert config(BWD, 8192, 2048, 512, 32) == (3, 12, 160, 256)
    assert config(DW, 999, 640, 448, 7) == (2, 4, 128, 128)
    assert config(DW, 8192, 512, 2048, 32) == (2, 4, 128, 256)


def test_refusals():
    lib = gmm.load_library()
    c = gmm.TileConfig()
    ask = lambda op, M=100, K=128, N=64, G=4, out=1, cfg=ctypes.byref(c): lib.gmm_get_tile_config(op, M, K, N, G, 1,
                                                                                                 out, cfg)
    for op in (FWD, BWD, DW):
        assert ask(op) == 0
        assert ask(op, cfg=None) == NULL
        assert ask(op, out=2) == DTYPE
        for kw in (dict(M=0), dict(M=-1), dict(K=96), dict(N=32), dict(N=1 << 30), dict(G=0), dict(G=5000)):
            assert ask(op, **kw) == SHAPE, kw
    assert ask(19) == SHAPE and ask(15) == SHAPE
