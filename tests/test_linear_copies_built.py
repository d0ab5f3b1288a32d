"""The written-out copies of the projections' tiled product, in the built
library: five wait states lie between a scalar register that a vector
instruction wrote (one kept in a vector register and read back among them) and
a buffer load that reads it.  The compiler adds them for the loads it knows of,
not for those in assembly."""
import os
import re
import struct
import subprocess

import pytest

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
WAIT = 5


def code_objects(path):
    """The gfx950 code objects of a library's offload bundles."""
    data = open(path, "rb").read()
    magic = b"__CLANG_OFFLOAD_BUNDLE__"
    at = data.find(magic)
    while at >= 0:
        n, p = struct.unpack_from("<Q", data, at + len(magic))[0], at + len(magic) + 8
        for _ in range(n):
            off, size, name = struct.unpack_from("<QQQ", data, p)
            if size and b"gfx950" in data[p + 24:p + 24 + name]:
                yield data[at + off:at + off + size]
            p += 24 + name
        at = data.find(magic, at + 1)


def scalars(operand):
    m = re.match(r"s\[(\d+):(\d+)\]$|s(\d+)$", operand)
    if not m:
        return set()
    return set(range(int(m[1]), int(m[2]) + 1)) if m[1] else {int(m[3])}


def instructions(text):
    """(address, mnemonic, operands, branch target) of a listing, and the functions' addresses."""
    out, symbols = [], {}
    for line in text.splitlines():
        m = re.match(r"([0-9a-f]+) <(\S+)>:$", line)
        if m:
            symbols[m[2]] = int(m[1], 16)
            continue
        m = re.match(r"\t(\S+)\s*(.*?)\s*// ([0-9A-F]+):.*?(?:<(\S+?)(?:\+0x([0-9a-f]+))?>)?$", line)
        if m:
            out.append((int(m[3], 16), m[1], re.split(r"[,\s]+", m[2]), (m[4], int(m[5] or "0", 16)) if m[4] else None))
    return out, symbols


def too_near(code, symbols):
    """Loads to LDS within WAIT states after a vector instruction's write of a
    scalar they read, along the code's order and along its jumps; and how many
    such loads there are."""
    index = {c[0]: i for i, c in enumerate(code)}

    def reads_soon(i, states, written, jumps):
        while i < len(code) and states < WAIT:
            _, op, args, target = code[i]
            if op.startswith("buffer_load") and "lds" in args and written & scalars(args[1]):
                return code[i]
            if target and jumps and target[0] in symbols:
                hit = reads_soon(index[symbols[target[0]] + target[1]], states + 1, written, jumps - 1)
                if hit:
                    return hit
            if op in ("s_branch", "s_endpgm", "s_setpc_b64"):
                return None
            states += int(args[0], 0) + 1 if op == "s_nop" else 1
            i += 1
        return None

    bad, loads = [], 0
    for i, (_, op, args, _) in enumerate(code):
        loads += op.startswith("buffer_load") and "lds" in args
        written = scalars(args[0]) if op.startswith("v_") else set()
        if "_co_" in op or op.startswith(("v_div_scale", "v_mad_u64", "v_mad_i64")):      # carries
            written = written | scalars(args[1])
        if written:
            hit = reads_soon(i + 1, 0, written, 3)
            if hit:
                bad.append((code[i], hit))
    return bad, loads


def test_listing_is_understood():
    """The search finds what it looks for: in order, over a jump, and not past the wait."""
    def listing(*ops):
        return "0000000000000100 <f>:\n" + "\n".join(f"\t{o} // {0x100 + 4 * i:012X}: 00000000" + t for i, (o, t) in enumerate(ops))
    load = ("buffer_load_dwordx4 v2, s[8:11], 0 offen lds", "")
    write, nop = ("v_readlane_b32 s9, v1, 3", ""), ("s_nop 4", "")
    for ops, n in (((write, load), 1), ((write, nop, load), 0), ((write, ("s_nop 3", ""), load), 1),
                   ((("v_readlane_b32 s12, v1, 3", ""), load), 0),
                   ((load, nop, write, ("s_cbranch_scc1 65532", " <f>"), nop), 1)):
        bad, loads = too_near(*instructions(listing(*ops)))
        assert (len(bad), loads) == (n, 1), ops


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no disassembler")
def test_copies_do_not_follow_their_descriptors_too_soon(tmp_path):
    from sparse_output_layer_amd import haste
    haste.lib()
    seen = 0
    for n, blob in enumerate(code_objects(haste.LIB_PATH)):
        if b"k_linear_tile" not in blob:
            continue
        path = tmp_path / f"{n}.co"
        path.write_bytes(blob)
        text = subprocess.run([OBJDUMP, "-d", str(path)], check=True, capture_output=True, text=True).stdout
        bad, loads = too_near(*instructions(text))
        assert not bad, bad[:5]
        seen += loads
    assert seen > 1000
