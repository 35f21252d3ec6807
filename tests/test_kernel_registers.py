"""Register allocation of kernels whose matrix instructions are inline asm: a
register spilled or reloaded around them is traffic that the waits counted by
hand in those kernels know nothing of.  Read from the metadata that the
compiler wrote into the built library; nothing is run."""
import re
import struct

import msgpack
import pytest

import moe_grouped_gemm_gmm_amd as gmm

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def device_objects(data):
    """The gfx950 code objects bundled in the library."""
    for m in re.finditer(re.escape(MAGIC), data):
        base = m.start()
        (n,) = struct.unpack_from("<Q", data, base + len(MAGIC))
        at = base + len(MAGIC) + 8
        if n > 16:
            continue
        for _ in range(n):
            off, size, idlen = struct.unpack_from("<QQQ", data, at)
            name = data[at + 24:at + 24 + idlen]
            at += 24 + idlen
            if b"gfx950" in name and size:
                yield data[base + off:base + off + size]


def kernels(obj):
    """Kernel metadata of one code object (an ELF file with a msgpack note)."""
    (shoff,) = struct.unpack_from("<Q", obj, 0x28)
    entsize, num = struct.unpack_from("<HH", obj, 0x3A)
    for i in range(num):
        kind = struct.unpack_from("<I", obj, shoff + i * entsize + 4)[0]
        off, size = struct.unpack_from("<QQ", obj, shoff + i * entsize + 24)
        if kind != 7:                                     # SHT_NOTE
            continue
        at, end = off, off + size
        while at + 12 <= end:
            nlen, dlen, ntype = struct.unpack_from("<III", obj, at)
            name = obj[at + 12:at + 12 + nlen].rstrip(b"\0")
            at += 12 + (nlen + 3) // 4 * 4
            if name == b"AMDGPU" and ntype == 32:
                for k in msgpack.unpackb(obj[at:at + dlen], strict_map_key=False)["amdhsa.kernels"]:
                    yield k
            at += (dlen + 3) // 4 * 4


@pytest.fixture(scope="module")
def all_kernels():
    gmm.load_library()
    with open(gmm.LIB_PATH, "rb") as f:
        return {k[".name"]: k for o in device_objects(f.read()) for k in kernels(o)}


def test_load_wave_kernels_keep_everything_in_registers(all_kernels):
    ws = {n: k for n, k in all_kernels.items() if "ffn_ws_kernel" in n}
    assert len(ws) == 8            # forward: 3 kinds of kept P x 2 output types; dX: 2 output types
    for n, k in ws.items():
        assert k[".vgpr_spill_count"] == 0 and k[".private_segment_fixed_size"] == 0, n
