"""Register allocation of the plain forward on load-wave tiles: its kernels run
the body of the gated block's, whose matrix instructions are inline asm with
waits counted by hand, under a name of their own."""
from test_kernel_registers import all_kernels  # noqa: F401  (a fixture)


def test_plain_load_wave_kernels_keep_everything_in_registers(all_kernels):  # noqa: F811
    ws = {n: k for n, k in all_kernels.items() if "linear_ws_kernel" in n}
    assert len(ws) == 2            # two output types
    for n, k in ws.items():
        assert k[".vgpr_spill_count"] == 0 and k[".private_segment_fixed_size"] == 0, n


def test_every_kernel_of_that_body_is_looked_at(all_kernels):  # noqa: F811
    """Here or with the gated block's: a third name for it (768 threads, the products' arguments) would be missed."""
    names = [n for n, k in all_kernels.items() if "FfnArgs" in n and k[".max_flat_workgroup_size"] == 768]
    assert len(names) == 10 and all("ffn_ws_kernel" in n or "linear_ws_kernel" in n for n in names)
