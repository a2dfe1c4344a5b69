"""The wait states that loads need, read from the library's own code, without a GPU.

A memory instruction may read a scalar register five wait states after a vector instruction has written
it, and a load to LDS may read m0 one after its write.  The compiler sees to both for the instructions
that it places itself, but not inside inline assembly, and a load that comes too early takes an old
address, length or place in LDS now and then only.  So the code is disassembled and every way that leads
to such an instruction is walked back.  The code the library ships is the one that this reads.
"""
import os
import re
import struct
import subprocess

import pytest

import gated_delta_rule_gdn2_amd as gdn2

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
SGPR_WAIT, M0_WAIT = 5, 1


def code_objects(blob):
    """The gfx950 code objects of a library's offload bundles."""
    at = blob.find(MAGIC)
    while at >= 0:
        count, = struct.unpack_from("<Q", blob, at + 24)
        entry = at + 32
        for _ in range(count):
            off, size, n = struct.unpack_from("<QQQ", blob, entry)
            if size and b"gfx950" in blob[entry + 24:entry + 24 + n]:
                yield blob[at + off:at + off + size]
            entry += 24 + n
        at = blob.find(MAGIC, at + 24)


class Instr:
    __slots__ = ("text", "name", "ops", "addr", "before")

    def __init__(self, text, addr):
        self.text, self.addr, self.before = text, addr, []
        parts = text.split(None, 1)
        self.name, self.ops = parts[0], [o.strip() for o in parts[1].split(",")] if len(parts) > 1 else []


def functions(listing):
    """[(name, instructions)], each instruction with those that may come right before it."""
    out, by_addr = [], {}
    for line in listing.splitlines():
        head = re.match(r"^[0-9a-fA-F]{16} <(.+)>:$", line)
        if head:
            out.append((head.group(1), []))
            continue
        body = re.match(r"^\s+(\S.*?)\s*// ([0-9A-Fa-f]{12}):", line)
        if body:
            i = Instr(body.group(1), int(body.group(2), 16))
            out[-1][1].append(i)
            by_addr[i.addr] = i
    for _, code in out:
        last = None
        for i in code:
            if last is not None and not last.name.startswith(("s_branch", "s_endpgm", "s_setpc")):
                i.before.append(last)
            if i.name.startswith(("s_branch", "s_cbranch")):
                words = int(i.ops[0])  # behind the branch, signed
                by_addr[i.addr + 4 + 4 * (words - (words >> 15 << 16))].before.append(i)
            last = i
    return out


def scalars(op):
    """The scalar registers that an operand names."""
    op = op.split()[0] if op else ""
    if op == "vcc":
        return {"vcc_lo", "vcc_hi"}
    if op in ("vcc_lo", "vcc_hi", "m0"):
        return {op}
    one = re.match(r"^s(\d+)$", op)
    if one:
        return {int(one.group(1))}
    many = re.match(r"^s\[(\d+):(\d+)\]$", op)
    return set(range(int(many.group(1)), int(many.group(2)) + 1)) if many else set()


def scalars_written(i):
    if i.name.startswith("v_") and i.ops:
        if i.name.startswith("v_cmp") and i.name.endswith("_e32"):
            return {"vcc_lo", "vcc_hi"}
        written = scalars(i.ops[0])  # v_readfirstlane, v_readlane, v_cmp
        if not written and len(i.ops) > 2 and re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co_|v_mad_[iu]64|v_div_scale", i.name):
            written = scalars(i.ops[1])  # the carry or flag beside a vector result
        return written
    return set()


def is_memory(i):
    return i.name.startswith(("buffer_", "global_", "flat_", "scratch_")) and not i.name.startswith(("buffer_wbl2", "buffer_inv"))


def too_early(i, need, written):
    """A way back from i on which an instruction that `written` knows is fewer than `need` wait states away, or None."""
    seen, todo = {}, [(b, 0) for b in i.before]
    while todo:
        b, states = todo.pop()
        if seen.get(b.addr, need) <= states:
            continue
        seen[b.addr] = states
        if written(b):
            return b
        states += int(b.ops[0], 0) + 1 if b.name == "s_nop" else 1
        if states < need:
            todo += [(x, states) for x in b.before]
    return None


def faults(code):
    bad = []
    for i in code:
        if not is_memory(i):
            continue
        reads = set().union(set(), *(scalars(o) for o in i.ops))
        b = too_early(i, SGPR_WAIT, lambda x: scalars_written(x) & reads) if reads else None
        if b is not None:
            bad.append((b.text, i.text))
        if i.text.endswith(" lds") or "_lds_" in i.name:
            b = too_early(i, M0_WAIT, lambda x: x.name.startswith("s_") and bool(x.ops) and x.ops[0] == "m0")
            if b is not None:
                bad.append((b.text, i.text))
    return bad


def listing_of(text):
    lines = ["\t%s // %012X: 00000000" % (t, 4 * n) for n, t in enumerate(text.splitlines())]
    return "\n".join(["%016x <f>:" % 0] + lines)


LOAD = "buffer_load_dwordx4 v1, s[4:7], 0 offen lds"


@pytest.mark.parametrize("text,count", [
    ("s_mov_b32 m0, s3\n" + LOAD, 1),
    ("s_mov_b32 m0, s3\ns_nop 0\n" + LOAD, 0),
    ("v_readfirstlane_b32 s6, v1\ns_mov_b32 m0, s3\ns_nop 0\n" + LOAD, 1),
    ("v_readfirstlane_b32 s6, v1\ns_mov_b32 m0, s3\ns_nop 2\n" + LOAD, 1),
    ("v_readfirstlane_b32 s6, v1\ns_mov_b32 m0, s3\ns_nop 3\n" + LOAD, 0),
    ("v_readfirstlane_b32 s8, v1\ns_mov_b32 m0, s3\ns_nop 0\n" + LOAD, 0),
    ("v_cmp_lt_u32_e64 s[6:7], v1, v2\n" + LOAD, 1),
    ("v_add_co_u32_e64 v3, s[4:5], v1, v2\n" + LOAD, 1),
    ("v_readlane_b32 s9, v1, 3\nglobal_load_dword v1, v2, s[8:9]", 1),
    ("v_readfirstlane_b32 s6, v1\ns_cbranch_scc1 3\ns_nop 4\ns_nop 4\ns_nop 4\n" + LOAD, 1),  # past the waits
    ("v_readfirstlane_b32 s6, v1\ns_branch 1\nv_readfirstlane_b32 s6, v1\ns_nop 4\ns_nop 4\ns_nop 3\n" + LOAD, 0),
])
def test_the_walk_finds_what_it_should(text, count):
    (_, code), = functions(listing_of(text))
    assert len(faults(code)) == count


def test_loads_wait_for_their_scalar_registers(tmp_path):
    if not os.path.exists(gdn2.library_path()):
        pytest.skip("libgdn2.so not built")
    if not os.path.exists(OBJDUMP):
        pytest.skip("no disassembler")
    with open(gdn2.library_path(), "rb") as f:
        blob = f.read()
    bad, to_lds = [], 0
    for n, obj in enumerate(code_objects(blob)):
        path = tmp_path / ("%d.elf" % n)
        path.write_bytes(obj)
        text = subprocess.run([OBJDUMP, "-d", str(path)], capture_output=True, text=True, check=True).stdout
        for name, code in functions(text):
            to_lds += sum(1 for i in code if i.text.endswith(" lds") or "_lds_" in i.name)
            bad += [(name,) + f for f in faults(code)]
    assert to_lds > 0
    assert not bad, "%d of %d, the first: %s" % (len(bad), to_lds, bad[:3])
