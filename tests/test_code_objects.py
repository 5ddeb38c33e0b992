"""The gfx950 code of libmxq.so, disassembled: orders that the hardware asks
of a program and that the compiler does not see to inside inline assembly."""
import os
import re
import shutil
import struct
import subprocess

import pytest

from nvfp4_block_scaled_amax_amd import _binding

OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(blob):
    """The gfx950 images of every offload bundle in a library's bytes."""
    at = blob.find(MAGIC)
    while at >= 0:
        n, = struct.unpack_from("<Q", blob, at + len(MAGIC))
        p = at + len(MAGIC) + 8
        for _ in range(n):
            off, size, name = struct.unpack_from("<QQQ", blob, p)
            triple = blob[p + 24:p + 24 + name]
            p += 24 + name
            if b"gfx950" in triple and size:
                yield blob[at + off:at + off + size]
        at = blob.find(MAGIC, p)


def instructions(image, tmp_path):
    path = tmp_path / "image.o"
    path.write_bytes(image)
    r = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(path)], capture_output=True,
                       text=True, check=True)
    for line in r.stdout.splitlines():
        m = re.match(r"\s+([a-z]\w+)\s*([^/]*)", line)
        if m:
            yield m.group(1), m.group(2).strip()


def scalars(arg):
    """The scalar registers an operand names."""
    m = re.fullmatch(r"s(\d+)|s\[(\d+):(\d+)\]", arg)
    if not m:
        return set()
    lo = int(m.group(1) or m.group(2))
    return set(range(lo, int(m.group(3) or lo) + 1))


def unwaited(code):
    """Loads to LDS that directly follow a scalar write of M0, their base in
    LDS; loads to LDS within five wait states of a vector instruction's write
    of their scalar address; and how many loads to LDS there are."""
    bad, loads, past = [], 0, []          # past: the last five wait states
    for op, args in code:
        if op.startswith(("global_load_lds", "scratch_load_lds")) \
                or op.startswith("buffer_load") and args.endswith(" lds"):
            loads += 1
            if past and past[-1][0].startswith("s_") and re.match(r"m0\b", past[-1][1]):
                bad.append((past[-1], (op, args)))
            reads = set().union(*map(scalars, re.split(r"[ ,]+", args)))
            bad += [(p, (op, args)) for p in past if p[0].startswith("v_")
                    and scalars(p[1].split(",")[0]) & reads]
        waits = int(args, 0) + 1 if op == "s_nop" else 1
        past = (past + [(op, args)] * waits)[-5:]
    return bad, loads


def test_a_load_to_lds_waits_for_m0():
    assert unwaited([("s_mov_b32", "m0, s4"), ("global_load_lds_dword", "v1, s[0:1]")])[0]
    assert unwaited([("s_add_i32", "m0, s4, s5"), ("buffer_load_dword", "v1, s[0:3], 0 offen lds")])[0]
    assert unwaited([("s_mov_b32", "m0, s4"), ("s_nop", "0"),
                     ("global_load_lds_dword", "v1, s[0:1]")]) == ([], 1)


def test_a_load_to_lds_waits_for_its_scalar_address():
    lane, load = ("v_readlane_b32", "s1, v3, 0"), ("global_load_lds_dword", "v1, s[0:1]")
    assert unwaited([lane, load])[0]
    assert unwaited([lane, ("s_nop", "3"), load])[0]
    assert unwaited([lane, ("s_nop", "4"), load]) == ([], 1)
    assert unwaited([("v_readlane_b32", "s2, v3, 0"), load]) == ([], 1)


def test_library_loads_to_lds_wait_for_m0(tmp_path):
    """A scalar write of M0 needs one wait state before a load to LDS, which
    takes its address from it, and a vector instruction's write of a scalar
    register five before a load's address reads it."""
    if not os.path.exists(_binding.LIB_PATH) or not os.path.exists(OBJDUMP):
        pytest.skip("no built library, or no disassembler")
    with open(_binding.LIB_PATH, "rb") as f:
        blob = f.read()
    images = list(code_objects(blob))
    assert images
    bad, loads = [], 0
    for image in images:
        b, n = unwaited(instructions(image, tmp_path))
        bad += b
        loads += n
    assert loads > 100
    assert not bad, (len(bad), bad[0])
