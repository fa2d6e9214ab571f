"""The waits that the direct loads from memory into LDS need, in the device code
as it was built (no GPU).  Those loads are inline assembly: a scalar register
that a vector instruction wrote may be read by one no sooner than five wait states
later, and the compiler sees to that for its own instructions only.  Looks back
from every such load along all paths of its kernel."""

import collections
import os
import re
import shutil
import struct
import subprocess

import pytest

import collective_communication_reduction_way_amd as rr

WAITS = 5
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def device_objects(path):
    """The gfx950 code objects of a shared library."""
    with open(path, "rb") as f:
        blob = f.read()
    at = blob.find(MAGIC)
    while at >= 0:
        (count,) = struct.unpack_from("<Q", blob, at + len(MAGIC))
        pos = at + len(MAGIC) + 8
        for _ in range(count):
            offset, size, n = struct.unpack_from("<QQQ", blob, pos)
            name = blob[pos + 24:pos + 24 + n]
            pos += 24 + n
            if b"gfx950" in name and size:
                yield blob[at + offset:at + offset + size]
        at = blob.find(MAGIC, pos)


def scalars(operand):
    m = re.match(r"s\[(\d+):(\d+)\]$", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.match(r"s(\d+)$", operand)
    return {int(m[1])} if m else set()


class Kernel:
    def __init__(self, name):
        self.name, self.code, self.place = name, [], {}

    def add(self, line):
        # "<op> <operands> // <address>: <encoding> <target>"
        text, _, tail = line.partition("//")
        address = int(tail.split(":")[0], 16)
        op, _, rest = text.strip().partition(" ")
        target = re.search(r"<[^>]*\+0x([0-9a-f]+)>\s*$", tail)
        self.place[address] = len(self.code)
        self.code.append((op, [o.strip() for o in rest.split(",")], address,
                          int(target[1], 16) if target else 0 if tail.rstrip().endswith(">") else None))

    def short_waits(self):
        """(load, writer, wait states between) of every load that comes too soon, and the number of loads."""
        before = collections.defaultdict(list)
        base = self.code[0][2]
        for i, (op, _, _, target) in enumerate(self.code):
            if op.startswith(("s_branch", "s_cbranch")):
                before[self.place[base + target]].append(i)
            if not op.startswith(("s_branch", "s_endpgm", "s_setpc")):
                before[i + 1].append(i)
        found, loads = [], 0
        for i, (op, operands, _, _) in enumerate(self.code):
            if not (op.startswith("buffer_load") and operands[-1].endswith(" lds")):
                continue
            loads += 1
            descriptor, least, todo = scalars(operands[1]), {}, [(j, 0) for j in before[i]]
            assert len(descriptor) == 4, operands
            while todo:
                j, waits = todo.pop()
                if waits >= WAITS or least.get(j, WAITS) <= waits:
                    continue
                least[j] = waits
                o, args, _, _ = self.code[j]
                writes = scalars(args[0]) | (scalars(args[1]) if "_co_" in o and len(args) > 1 else set())
                if o.startswith("v_") and writes & descriptor:
                    found.append((" ".join(self.code[i][:1] + tuple(operands)), f"{o} {', '.join(args)}", waits))
                    continue
                waits += int(args[0], 0) + 1 if o == "s_nop" else 1
                todo += [(k, waits) for k in before[j]]
        return found, loads


def kernels(objdump, obj, tmp_path):
    path = tmp_path / "code.o"
    path.write_bytes(obj)
    text = subprocess.run([objdump, "-d", "--no-show-raw-insn", str(path)], capture_output=True, text=True, check=True).stdout
    kernel = None
    for line in text.splitlines():
        m = re.match(r"[0-9a-f]+ <(.*)>:$", line)
        if m:
            if kernel and kernel.code:
                yield kernel
            kernel = Kernel(m[1])
        elif kernel and "//" in line:
            kernel.add(line)
    if kernel and kernel.code:
        yield kernel


def test_descriptors_are_there_when_loads_read_them(tmp_path):
    objdump = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
    if not os.path.exists(objdump):
        pytest.skip("no llvm-objdump")
    loads = 0
    for obj in device_objects(rr.library_path()):
        if b"k_gated_hidden" not in obj and b"k_logits" not in obj:
            continue  # the kernels with direct loads
        for kernel in kernels(objdump, obj, tmp_path):
            found, n = kernel.short_waits()
            loads += n
            assert not found, (kernel.name, found)
    assert loads > 1000


def test_the_scan_sees_a_short_wait():
    kernel = Kernel("k")
    code = ["v_readfirstlane_b32 s6, v2", "s_branch 2 // 000000000104: 0 <k+0x10>", "s_nop 7", "s_nop 7",
            "s_add_u32 m0, s24, 0", "s_nop 0", "buffer_load_dwordx4 v55, s[4:7], 0 offen lds", "s_endpgm"]
    for i, line in enumerate(code):
        kernel.add(line if "//" in line else f"{line} // {0x100 + 4 * i:012x}:")
    found, loads = kernel.short_waits()
    assert loads == 1 and [(w, n) for _, w, n in found] == [("v_readfirstlane_b32 s6, v2", 3)]
