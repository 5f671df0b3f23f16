"""Registers of the selective scan's, the short convolution's and the norm's kernels, from the code objects in the
built library: none keeps vector registers in memory, and the gradients' kernels leave room for the waves a
SIMD that their sources name."""

import os
import re
import struct

import msgpack
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "linear_recurrence_rnn_amd", "liblinrec.so")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(data):
    """The gfx950 ELF images of the bundles in the library's bytes."""
    at = data.find(MAGIC)
    while at >= 0:
        count, pos = struct.unpack_from("<Q", data, at + len(MAGIC))[0], at + len(MAGIC) + 8
        for _ in range(count):
            offset, size, n = struct.unpack_from("<QQQ", data, pos)
            name = data[pos + 24:pos + 24 + n]
            pos += 24 + n
            if b"gfx950" in name and size:
                yield data[at + offset:at + offset + size]
        at = data.find(MAGIC, at + 1)


def kernels(elf):
    """The kernels' metadata: the note of type 32 in the image's PT_NOTE segments."""
    phoff, phsize, phnum = struct.unpack_from("<Q", elf, 32)[0], *struct.unpack_from("<HH", elf, 54)
    for i in range(phnum):
        kind, _, offset, _, _, size = struct.unpack_from("<IIQQQQ", elf, phoff + i * phsize)
        end = offset + size
        while kind == 4 and offset < end:
            namesz, descsz, note = struct.unpack_from("<III", elf, offset)
            desc = offset + 12 + (namesz + 3) // 4 * 4
            if note == 32:
                yield from msgpack.unpackb(elf[desc:desc + descsz], strict_map_key=False)["amdhsa.kernels"]
            offset = desc + (descsz + 3) // 4 * 4


@pytest.fixture(scope="module")
def found():
    if not os.path.exists(LIB):
        pytest.fail("liblinrec.so is not built (run python -m linear_recurrence_rnn_amd.build)")
    with open(LIB, "rb") as f:
        data = f.read()
    return {k[".name"]: k for elf in code_objects(data) for k in kernels(elf)}


@pytest.mark.parametrize("part,least", [("sel_", 40), ("short_conv", 65), ("rms_norm", 73)])
def test_nothing_in_memory(found, part, least):
    own = {n: k for n, k in found.items() if part in n}
    assert len(own) >= least
    for name, k in own.items():
        assert k[".vgpr_spill_count"] == 0 and k[".private_segment_fixed_size"] == 0, name


@pytest.mark.parametrize("waves,simd", [(1, 2), (2, 2), (4, 3)])
def test_waves_of_the_gradients(found, waves, simd):
    own = [(n, k) for n, k in found.items() if re.search("sel_gradient_kernelI.*Li%dELb" % waves, n)]
    assert len(own) == (4 if waves == 4 else 2)
    for name, k in own:
        total = k[".vgpr_count"]  # accumulation registers among them
        assert (total + 7) // 8 * 8 * simd <= 512, (name, total)
