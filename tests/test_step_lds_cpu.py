"""LDS of the built kernels of expert_step, from the code objects' own descriptions inside
the library that was built here from source."""
import os
import struct

import pytest

import spgemm_symbolic_row_amd as sg

msgpack = pytest.importorskip("msgpack")

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(data):
    """The ELF images for the GPU in a library with one bundle for each source file."""
    at = data.find(MAGIC)
    while at >= 0:
        count, = struct.unpack_from("<Q", data, at + len(MAGIC))
        entry = at + len(MAGIC) + 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, entry)
            name = data[entry + 24:entry + 24 + length]
            entry += 24 + length
            if b"gfx950" in name and size:
                yield data[at + offset:at + offset + size]
        at = data.find(MAGIC, entry)


def kernels(elf):
    """The kernels' descriptions: the note of type 32 of the name AMDGPU."""
    sections, = struct.unpack_from("<Q", elf, 40)
    size, count = struct.unpack_from("<HH", elf, 58)
    for i in range(count):
        kind, = struct.unpack_from("<I", elf, sections + i * size + 4)
        offset, length = struct.unpack_from("<QQ", elf, sections + i * size + 24)
        end = offset + length
        while kind == 7 and offset < end:
            names, descs, note = struct.unpack_from("<III", elf, offset)
            desc = offset + 12 + (names + 3) // 4 * 4
            if note == 32 and elf[offset + 12:offset + 18] == b"AMDGPU":
                return msgpack.unpackb(elf[desc:desc + descs])["amdhsa.kernels"]
            offset = desc + (descs + 3) // 4 * 4
    return []


def test_rows_of_x_begin_at_16_bytes():
    """The dynamic array begins where the static ones end: the host aligns x inside it to 16 bytes, so it has to begin at
    a multiple of those; and the static ones have to leave what the host counts on."""
    sg.lib()
    with open(os.path.join(os.path.dirname(sg.__file__), "libspgemm.so"), "rb") as f:
        found = [k for elf in code_objects(f.read()) for k in kernels(elf)]
    step = [k for k in found if "k_step" in k[".name"] and "StepArgs" in k[".name"]]
    assert len(step) == 16   # two types of x, two of the weights, four shapes of the routing
    for k in step:
        assert k[".group_segment_fixed_size"] % 16 == 0, k[".name"]
        assert k[".group_segment_fixed_size"] <= 46 * 1024
        assert k[".private_segment_fixed_size"] == 0 and k[".vgpr_spill_count"] == 0
