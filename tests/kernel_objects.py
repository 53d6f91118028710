"""The kernels in the built library, as its gfx950 code objects describe them
(the metadata notes that the compiler writes for the runtime)."""
import re
import struct

import msgpack

BUNDLE = b"__CLANG_OFFLOAD_BUNDLE__"


def _code_objects(data: bytes):
    """The gfx950 ELF images in the library's bundles."""
    at = data.find(BUNDLE)
    while at >= 0:
        count, = struct.unpack_from("<Q", data, at + len(BUNDLE))
        p = at + len(BUNDLE) + 8
        if count < 16:  # (the name can stand alone, as a text of the runtime's)
            for _ in range(count):
                offset, size, n = struct.unpack_from("<QQQ", data, p)
                if b"gfx950" in data[p + 24:p + 24 + n]:
                    yield data[at + offset:at + offset + size]
                p += 24 + n
        at = data.find(BUNDLE, at + len(BUNDLE))


def _notes(elf: bytes):
    """(type, contents) of the note sections' entries."""
    offset, = struct.unpack_from("<Q", elf, 0x28)
    size, count = struct.unpack_from("<HH", elf, 0x3A)
    for i in range(count):
        _, kind, _, _, at, n = struct.unpack_from("<IIQQQQ", elf, offset + i * size)
        if kind != 7:  # SHT_NOTE
            continue
        end = at + n
        while at + 12 <= end:
            name, length, what = struct.unpack_from("<III", elf, at)
            at += 12 + (name + 3) // 4 * 4
            yield what, elf[at:at + length]
            at += (length + 3) // 4 * 4


def kernels(path: str):
    """Mangled name -> the compiler's description of each kernel."""
    with open(path, "rb") as f:
        data = f.read()
    out = {}
    for elf in _code_objects(data):
        for what, text in _notes(elf):
            if what == 32:  # NT_AMDGPU_METADATA
                for k in msgpack.unpackb(text, strict_map_key=False)["amdhsa.kernels"]:
                    out[k[".name"]] = k
    return out


def instances(path: str, name: str):
    """The whole-number and truth-value arguments of each instance of a kernel
    template, as tuples."""
    found = set()
    for k in kernels(path):
        m = re.search(r"\d" + name + r"I((?:L[bi]\d+E)+)E", k)
        if m:
            found.add(tuple(int(x) for x in re.findall(r"L[bi](\d+)E", m.group(1))))
    return found
