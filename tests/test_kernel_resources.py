"""What the compiler took for the kernels, from the metadata in the built
library (no GPU): blocks that launch rules count two to a CU fit twice into its
160 KiB of LDS, and the products' kernels spill nothing to memory."""
import struct

import pytest

from combine_dispatch_layout_02_amd import ep

msgpack = pytest.importorskip("msgpack")
LDS = 160 * 1024


def _code_objects(data):
    """The gfx950 ELF files in the library's offload bundles."""
    magic, at = b"__CLANG_OFFLOAD_BUNDLE__", 0
    while (at := data.find(magic, at)) >= 0:
        n, = struct.unpack_from("<Q", data, at + 24)
        p = at + 32
        for _ in range(n if n < 16 else 0):
            off, size, length = struct.unpack_from("<QQQ", data, p)
            target = data[p + 24:p + 24 + length]
            p += 24 + length
            if b"gfx950" in target and size:
                yield data[at + off:at + off + size]
        at += len(magic)


def _kernels():
    """Metadata of every kernel, by its mangled name."""
    found = {}
    with open(ep.LIB_PATH, "rb") as f:
        data = f.read()
    for elf in _code_objects(data):
        phoff, = struct.unpack_from("<Q", elf, 32)
        size, count = struct.unpack_from("<HH", elf, 54)
        for i in range(count):
            kind, _, off, _, _, length = struct.unpack_from("<IIQQQQ", elf, phoff + i * size)
            if kind != 4:   # a note
                continue
            end = off + length
            while off + 12 <= end:
                name, desc, tag = struct.unpack_from("<III", elf, off)
                body = off + 12 + (name + 3) // 4 * 4
                if tag == 32 and elf[off + 12:off + 18] == b"AMDGPU":
                    for k in msgpack.unpackb(elf[body:body + desc])["amdhsa.kernels"]:
                        found[k[".name"]] = k
                off = body + (desc + 3) // 4 * 4
    return found


@pytest.fixture(scope="module")
def kernels():
    ep.load()
    found = _kernels()
    assert found
    return found


def _named(kernels, part):
    some = [k for name, k in kernels.items() if part in name]
    assert some, part
    return some


def test_two_blocks_a_cu(kernels):
    for part in ("ep_linear_gradients_kernel", "ep_few_up_kernel"):
        for k in _named(kernels, part):
            assert 2 * k[".group_segment_fixed_size"] <= LDS, k[".name"]


@pytest.mark.parametrize("part", ["ep_linear_", "ep_few_"])
def test_no_scratch(kernels, part):
    for k in _named(kernels, part):
        assert k[".group_segment_fixed_size"] <= LDS
        assert k[".private_segment_fixed_size"] == 0, k[".name"]
