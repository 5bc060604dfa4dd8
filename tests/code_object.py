"""What the compiler noted about the kernels of a built library: {name: {".group_segment_fixed_size":
LDS bytes, ".vgpr_spill_count": ...}} from the metadata of its gfx950 code objects."""
import struct

import msgpack


def _notes(elf):
    """The payloads of the AMDGPU metadata notes (type 32) of an ELF64 file."""
    at, size, count = (struct.unpack_from("<Q", elf, 40)[0], *struct.unpack_from("<HH", elf, 58))
    for i in range(count):
        kind, = struct.unpack_from("<I", elf, at + i * size + 4)
        begin, length = struct.unpack_from("<QQ", elf, at + i * size + 24)
        while kind == 7 and length > 12:
            name, desc, note = struct.unpack_from("<III", elf, begin)
            body = begin + 12 + (name + 3) // 4 * 4
            if note == 32:
                yield elf[body:body + desc]
            step = body + (desc + 3) // 4 * 4 - begin
            begin, length = begin + step, length - step


def kernels(path):
    with open(path, "rb") as f:
        data = f.read()
    magic, got, at = b"__CLANG_OFFLOAD_BUNDLE__", {}, 0
    while (at := data.find(magic, at)) >= 0:
        count, = struct.unpack_from("<Q", data, at + 24)
        p = at + 32
        for _ in range(count):
            begin, length, name = struct.unpack_from("<QQQ", data, p)
            if b"gfx950" in data[p + 24:p + 24 + name]:
                for note in _notes(data[at + begin:at + begin + length]):
                    for k in msgpack.unpackb(note)["amdhsa.kernels"]:
                        got[k[".name"]] = k
            p += 24 + name
        at += len(magic)
    return got
