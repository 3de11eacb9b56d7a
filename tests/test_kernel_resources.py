"""Registers of kernels whose time goes by the waves that hide their loads, as the
built library's own metadata states them (CPU only)."""
import os
import struct

import pytest

from kronecker_factored_second_amd import okls

msgpack = pytest.importorskip("msgpack")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _code_objects(data):
    """The gfx950 ELF files of every offload bundle in the library."""
    at = data.find(MAGIC)
    while at >= 0:
        entry = at + len(MAGIC) + 8
        for _ in range(struct.unpack_from("<Q", data, entry - 8)[0]):
            offset, size, length = struct.unpack_from("<QQQ", data, entry)
            if b"gfx950" in data[entry + 24: entry + 24 + length]:
                yield data[at + offset: at + offset + size]
            entry += 24 + length
        at = data.find(MAGIC, at + 1)


def _kernels(elf):
    """The kernels' entries in the metadata note (type 32, name AMDGPU) of one code object."""
    start, = struct.unpack_from("<Q", elf, 40)
    size, count = struct.unpack_from("<HH", elf, 58)
    for i in range(count):
        kind, = struct.unpack_from("<I", elf, start + i * size + 4)
        at, length = struct.unpack_from("<QQ", elf, start + i * size + 24)
        end = at + length
        while kind == 7 and at < end:
            name, desc, note = struct.unpack_from("<III", elf, at)
            body = at + 12 + (name + 3) // 4 * 4
            if note == 32 and elf[at + 12: at + 18] == b"AMDGPU":
                yield from msgpack.unpackb(elf[body: body + desc])["amdhsa.kernels"]
            at = body + (desc + 3) // 4 * 4


@pytest.fixture(scope="module")
def kernels():
    if not os.path.exists(okls.LIB_PATH):
        pytest.skip("libokls.so not built")
    with open(okls.LIB_PATH, "rb") as f:
        found = {k[".name"]: k for elf in _code_objects(f.read()) for k in _kernels(elf)}
    if not found:
        pytest.skip("the library's code objects are not laid out as plain bundles")
    return found


def _waves(kernel):
    """Waves a SIMD: 512 vector registers a lane, given out by eights, at most 8 waves."""
    return min(8, 512 // -(-kernel[".vgpr_count"] // 8 * 8))


# rows of 16, columns of 16, fp32 result: waves a SIMD
@pytest.mark.parametrize("tm,tn,f32,waves", [(1, 1, 0, 8), (1, 1, 1, 6), (2, 1, 0, 5), (2, 1, 1, 6)])
def test_few_rows_keep_their_waves(kernels, tm, tn, f32, waves):
    """The dense product of few rows reads the weight straight into registers, and waves are what has its loads in flight."""
    some = [k for n, k in kernels.items() if f"matmul_few_kernelILi{tm}ELi{tn}E" in n and n.split("EEEv")[0].endswith(f"Lb{f32}")]
    assert len(some) == 4           # both formats of both operands
    for k in some:
        assert _waves(k) >= waves and k[".vgpr_spill_count"] == 0 and k[".private_segment_fixed_size"] == 0, k[".name"]
