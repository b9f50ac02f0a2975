"""What the instruction set asks of code that no compiler checks (inline assembly),
read from the built library's own instructions (no GPU)."""

import os
import re
import subprocess

import pytest

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
SGPR = re.compile(r"\b(?:s(\d+)\b|s\[(\d+):(\d+)\]|(vcc)\b)")
SECOND = re.compile(r"v_(add|sub|subrev|addc|subb|subbrev)(_co)?_u32|v_(add|sub|subrev|addc|subb|subbrev)_co_|v_div_scale|v_mad_[ui]64_")


def sgprs(text):
    out = set()
    for one, lo, hi, vcc in SGPR.findall(text):
        out |= {"vcc"} if vcc else {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return out


def parse(listing):
    """Functions of a listing as [(address, mnemonic, operands)]."""
    functions, now = {}, None
    for line in listing.splitlines():
        head = re.match(r"^[0-9a-f]+ <(.+)>:$", line)
        if head:
            now = functions.setdefault(head.group(1), [])
            continue
        m = re.match(r"^\s+([a-z]\S*)\s*(.*?)\s*// ([0-9A-F]+):", line)
        if m and now is not None:
            now.append((int(m.group(3), 16), m.group(1), m.group(2)))
    return functions


def short_waits(code):
    """Vector-memory instructions that read a scalar register fewer than 5 wait states after a vector instruction wrote
    it, over every way there: [(address, states)]. (An instruction is one state, s_nop n is n + 1.)"""
    at = {address: n for n, (address, *_) in enumerate(code)}
    before = [[] for _ in code]
    for n, (address, op, args) in enumerate(code):
        if n + 1 < len(code) and op not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            before[n + 1].append(n)
        if op == "s_branch" or op.startswith("s_cbranch"):
            to = address + 4 + 4 * ((int(args.split()[0]) + (1 << 15)) % (1 << 16) - (1 << 15))
            if to in at:
                before[at[to]].append(n)

    def written(n):
        _, op, args = code[n]
        if not op.startswith("v_"):
            return set()
        parts = args.split(",")
        dst = sgprs(parts[0])
        if len(parts) > 1 and SECOND.match(op):
            dst |= sgprs(parts[1])
        return dst

    found = []
    for n, (address, op, args) in enumerate(code):
        if not op.startswith(("global_", "buffer_", "scratch_", "flat_")):
            continue
        need = sgprs(args)
        if not need:
            continue
        ways, least = [(n, 0, need)], 5
        while ways:
            k, states, regs = ways.pop()
            for p in before[k]:
                if regs & written(p):
                    least = min(least, states)
                    continue
                op_p, args_p = code[p][1], code[p][2]
                more = int(args_p.split()[0], 0) + 1 if op_p == "s_nop" else 1
                # what a scalar instruction writes afterwards is not the vector instruction's any more
                left = regs - sgprs(args_p.split(",")[0]) if op_p.startswith("s_") and "cmp" not in op_p else regs
                if states + more < 5 and left:
                    ways.append((p, states + more, left))
        if least < 5:
            found.append((address, least))
    return found


def test_short_waits_are_seen():
    text = """
0000000000001000 <f>:
	v_readfirstlane_b32 s10, v1                                // 000000001000: 00000000
	s_mov_b32 m0, s4                                           // 000000001004: 00000000
	s_nop {}                                                    // 000000001008: 00000000
	global_load_lds_dwordx4 v7, s[10:11]                       // 00000000100C: 00000000 00000000
	s_cbranch_scc1 65531                                       // 000000001014: 00000000 <f+0x4>
	s_endpgm                                                   // 000000001018: 00000000
"""
    for nop, want in ((0, [(0x100c, 2)]), (2, [(0x100c, 4)]), (3, [])):
        assert short_waits(parse(text.format(nop))["f"]) == want
    around = """
0000000000001000 <f>:
	global_load_lds_dwordx4 v7, s[10:11]                       // 000000001000: 00000000 00000000
	v_readfirstlane_b32 s11, v1                                // 000000001008: 00000000
	s_branch 65532                                             // 00000000100C: 00000000 <f>
"""
    assert short_waits(parse(around)["f"]) == [(0x1000, 1)]


def test_scalar_bases_of_copies_are_waited_for(tmp_path):
    """A scalar register that a vector instruction wrote is read by a vector-memory one 5 wait states later at the
    earliest: the hardware does not check it, and the compiler counts no instructions inside inline assembly."""
    from matrix_optimizer_step_02_amd import native
    if not os.path.exists(native.LIB_PATH) or not os.path.exists(OBJDUMP):
        pytest.skip("libmatopt.so not built, or no llvm-objdump")
    link = tmp_path / "lib.so"
    link.symlink_to(native.LIB_PATH)
    subprocess.run([OBJDUMP, "--offloading", str(link)], check=True, capture_output=True)
    images = sorted(p for p in tmp_path.iterdir() if "amdgcn" in p.name)
    assert images
    bad, copies = [], 0
    for image in images:
        out = subprocess.run([OBJDUMP, "-d", str(image)], check=True, capture_output=True, text=True).stdout
        for name, code in parse(out).items():
            copies += sum(op.startswith("global_load_lds") for _, op, *_ in code)
            bad += [(name, hex(address), states) for address, states in short_waits(code)]
    assert copies > 1000
    assert not bad, f"{len(bad)} sites, the first: {bad[:5]}"


def test_inline_assembly_names_what_it_writes():
    """A statement that writes m0 says so: a compiler that holds a value of its own there would not know."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "matrix_optimizer_step_02_amd", "csrc")
    seen = 0
    for name in sorted(os.listdir(csrc)):
        for statement in re.findall(r"\basm volatile\((.*?)\);", open(os.path.join(csrc, name)).read(), flags=re.S):
            if "m0," in statement.split("::")[0]:
                seen += 1
                assert '"m0"' in statement, f"{name}: {statement}"
    assert seen == 3
