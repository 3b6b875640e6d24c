"""The built library's kernels as the compiler describes them (its code objects' metadata): no GPU needed."""
import struct

import pytest

import overlap_tiling_trapezoidal_amd as tdp

msgpack = pytest.importorskip("msgpack")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
NT_AMDGPU_METADATA = 32


def code_objects(data):
    """The gfx950 ELF files bundled in a library."""
    at = data.find(MAGIC)
    while at >= 0:
        count, p = struct.unpack_from("<Q", data, at + len(MAGIC))[0], at + len(MAGIC) + 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            name = data[p + 24:p + 24 + length].decode()
            p += 24 + length
            if name.endswith("gfx950"):
                yield data[at + offset:at + offset + size]
        at = data.find(MAGIC, at + 1)


def kernels(elf):
    """A code object's kernels, by the note that holds their metadata."""
    assert elf[:5] == b"\x7fELF\x02"
    first, = struct.unpack_from("<Q", elf, 32)
    size, count = struct.unpack_from("<HH", elf, 54)
    for i in range(count):
        kind, _, offset, _, _, length = struct.unpack_from("<IIQQQQ", elf, first + i * size)
        if kind != 4:   # PT_NOTE
            continue
        p = offset
        while p < offset + length:
            names, desc, note = struct.unpack_from("<III", elf, p)
            body = p + 12 + (names + 3) // 4 * 4
            if note == NT_AMDGPU_METADATA:
                yield from msgpack.unpackb(elf[body:body + desc], strict_map_key=False)["amdhsa.kernels"]
            p = body + (desc + 3) // 4 * 4


@pytest.mark.device_abi
def test_products_keep_their_registers():
    """A product's loop waits for its operands' loads by their number, which a register read back from memory joins:
    none is spilled."""
    with open(tdp.LIB_PATH, "rb") as f:
        found = [k for elf in code_objects(f.read()) for k in kernels(elf) if "product_kernel" in k[".name"]]
    assert len(found) >= 15
    for k in found:
        assert k[".vgpr_spill_count"] == 0 and k[".private_segment_fixed_size"] == 0, k[".name"]
