"""What the loads to LDS of latent attention take for granted and the compiler does
not see to, since they are written as instructions, checked in the built library
(our own build, disassembled).

A buffer instruction may read a scalar register that a vector instruction wrote
(v_readlane, v_readfirstlane, a comparison) only five wait states later; an
instruction is one, s_nop N is N + 1.  Between m0 being written and a load to LDS
stands one.  Both over every path that leads to the load.  And m0 is those loads'
alone: each writes it for itself, and no other instruction has it.

The ring's waits count loads: before the barrier of a step the newest may still be under
way, as many as the wait names.  That is right if at least so many loads belong to
later steps, that is, if on every path from one such wait to the next a step's loads
are issued.  (Not for latent_expanded_kernel, which has two copies of a step's loads, one for
waves that see none of its keys: the compiler tests that condition twice, so that
paths exist with both copies and with neither that no wave takes.)
"""
import os
import re
import subprocess
import tempfile

import pytest

import latency_skinny_gemm_amd as skg
from latency_skinny_gemm_amd import build as lib_build
from tests.test_isa_cpu import LLVM, _gfx950_objects

KERNELS = ("latent_attention_kernel", "latent_expanded_kernel", "heads_ring_kernel")
WAIT = 5    # wait states from a vector instruction's scalar result to a buffer instruction
M0_WAIT = 1  # and from m0 to a load to LDS


def parse(lines):
    """[(mnemonic, operands, target offset or None, offset)] of one function's lines of (offset, text, target)."""
    out = []
    for offset, text, target in lines:
        name, _, rest = text.partition(" ")
        out.append((name, [o.strip() for o in rest.split(",")] if rest else [], target, offset))
    return out


def scalars(operand):
    """The scalar registers that an operand names, as a set of numbers (vcc as 1000, 1001, m0 as 1002)."""
    m = re.match(r"^s\[(\d+):(\d+)\]$", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.match(r"^s(\d+)$", operand)
    if m:
        return {int(m.group(1))}
    return {"vcc": {1000, 1001}, "vcc_lo": {1000}, "vcc_hi": {1001}, "m0": {1002}}.get(operand, set())


def written_by_vector(name, ops):
    """Scalar registers that a vector instruction writes: its first operand, and a carry's, which is its second."""
    if not name.startswith("v_") or not ops:
        return set()
    got = scalars(ops[0])
    if re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co_|v_div_scale|v_mad_[iu]64", name) and len(ops) > 1:
        got = got | scalars(ops[1])
    return got


def states(name, ops):
    return int(ops[0], 0) + 1 if name == "s_nop" else 1


def before(code):
    """For every instruction, those that may run right before it."""
    at = {offset: i for i, (_, _, _, offset) in enumerate(code)}
    prev = [[] for _ in code]
    for i, (name, _, target, _) in enumerate(code):
        if i + 1 < len(code) and name not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            prev[i + 1].append(i)
        if target is not None and target in at:
            prev[at[target]].append(i)
    return prev


def too_close(code, prev, i, registers, writes, wait):
    """An instruction that writes one of the registers fewer than `wait` states before number i, on any path; or None."""
    todo, best = [(p, 0) for p in prev[i]], {}
    while todo:
        p, passed = todo.pop()
        if passed >= wait or best.get(p, wait) <= passed:
            continue
        best[p] = passed
        name, ops, _, _ = code[p]
        if writes(name, ops) & registers:
            return p
        passed += states(name, ops)
        todo += [(q, passed) for q in prev[p]]
    return None


def hazards(code):
    """Descriptions of the places where a buffer instruction follows too soon."""
    prev, found = before(code), []
    for i, (name, ops, _, offset) in enumerate(code):
        if not name.startswith("buffer_") or name in ("buffer_wbl2", "buffer_inv"):
            continue
        lds = any(re.search(r"\blds\b", o) for o in ops)
        regs = set().union(*(scalars(o.split()[0]) for o in ops if o))
        p = too_close(code, prev, i, regs, written_by_vector, WAIT)
        if p is not None:
            found.append(f"{code[p][0]} {', '.join(code[p][1])} before {name} {', '.join(ops)} at {offset:#x}")
        if lds:
            p = too_close(code, prev, i, {1002}, lambda n, o: scalars(o[0]) if o and not n.startswith("s_cmp") else set(), M0_WAIT)
            if p is not None:
                found.append(f"m0 of {code[p][0]} right before {name} at {offset:#x}")
    return found


def others_with_m0(code):
    """Instructions with m0 that are no load's own addition, and loads to LDS without one."""
    found, own = [], set()
    for i, (name, ops, _, offset) in enumerate(code):
        if any(re.search(r"\blds\b", o) for o in ops):
            made = i >= 2 and code[i - 1][0] == "s_nop" and code[i - 2][0] == "s_add_u32" and code[i - 2][1][0] == "m0"
            if made:
                own.add(i - 2)
            else:
                found.append(f"{name} at {offset:#x}")
    for i, (name, ops, _, offset) in enumerate(code):
        implicit = re.match(r"s_movrel|v_movrel|ds_gws|ds_ordered|s_sendmsg|s_set_gpr", name)
        if (implicit or any(o == "m0" for o in ops)) and i not in own:
            found.append(f"{name} {', '.join(ops)} at {offset:#x}")
    return found


@pytest.fixture(scope="module")
def functions():
    for tool in ("llvm-objcopy", "llvm-objdump"):
        if not os.path.exists(os.path.join(LLVM, tool)):
            pytest.skip(f"{tool} not installed")
    if not os.path.exists(skg.library_path()):
        lib_build.build()
    funcs = {}
    with tempfile.TemporaryDirectory() as d:
        fb = os.path.join(d, "fatbin")
        subprocess.run([os.path.join(LLVM, "llvm-objcopy"), "--dump-section", f".hip_fatbin={fb}", skg.library_path()], check=True)
        for n, co in enumerate(_gfx950_objects(open(fb, "rb").read())):
            if not any(k.encode() in co for k in KERNELS):
                continue
            path = os.path.join(d, f"co{n}.o")
            open(path, "wb").write(co)
            dis = subprocess.run([os.path.join(LLVM, "llvm-objdump"), "-d", "--mcpu=gfx950", path], check=True, capture_output=True, text=True).stdout
            cur, start = None, 0
            for line in dis.splitlines():
                m = re.match(r"^([0-9a-f]+) <(\S+)>:\s*$", line)
                if m:
                    cur, start = m.group(2), int(m.group(1), 16)
                    funcs[cur] = []
                elif cur is not None and line.startswith("\t"):
                    text, _, comment = line.partition("//")
                    addr = re.match(r"\s*([0-9A-Fa-f]+):", comment)
                    if addr is None:  # the "..." that stands for a run of zero words
                        continue
                    tgt = re.search(r"<[^>+]*\+0x([0-9a-f]+)>", comment)
                    funcs[cur].append((int(addr.group(1), 16) - start, text.strip(), int(tgt.group(1), 16) if tgt else None))
    return {name: parse(lines) for name, lines in funcs.items()}


def test_every_kernel_is_there(functions):
    for kernel, n in zip(KERNELS, (4, 1, 4)):
        assert sum(kernel in name for name in functions) == n, kernel


def test_scalar_operands_have_settled(functions):
    loads = 0
    for name, code in functions.items():
        if any(k in name for k in KERNELS):
            here = sum(c[0] == "buffer_load_dwordx4" and any(re.search(r"\blds\b", o) for o in c[1]) for c in code)
            assert here > 0, name
            loads += here
            assert hazards(code) == [], name
    assert loads > 100


def test_m0_is_the_loads_own(functions):
    for name, code in functions.items():
        if any(k in name for k in KERNELS):
            assert others_with_m0(code) == [], name


def is_lds_load(name, ops):
    return name.startswith("buffer_load") and any(re.search(r"\blds\b", o) for o in ops)


def least_loads(code, start, ends):
    """The least number of loads to LDS on any path from behind instruction `start` to one of `ends`.  A branch around
    a load for waves without a lane that makes it is none: the lanes that make a step's last load are the first ones."""
    at = {offset: i for i, (_, _, _, offset) in enumerate(code)}
    best, todo, least = {}, [(0, start + 1)], None
    while todo:
        n, i = todo.pop()
        if i >= len(code) or best.get(i, n + 1) <= n:
            continue
        best[i] = n
        if i in ends:
            least = n if least is None else min(least, n)
            continue
        name, ops, target, _ = code[i]
        n += is_lds_load(name, ops)
        around = name == "s_cbranch_execz" and target in at and any(is_lds_load(*code[k][:2]) for k in range(i, at[target]))
        if target in at and not around:
            todo.append((n, at[target]))
        if name not in ("s_branch", "s_endpgm"):
            todo.append((n, i + 1))
    return least


def ring_waits(code, count):
    """Waits for all but `count` loads in front of a barrier."""
    return {i for i, (name, ops, _, _) in enumerate(code)
            if name == "s_waitcnt" and f"vmcnt({count})" in " ".join(ops) and code[i + 1][0] == "s_barrier"}


# kernel: loads of a step that a wave makes, and how many may be under way behind a step's wait
RINGS = {"latent_attention_kernelILi1ELi4ELb0E": (9, 9), "latent_attention_kernelILi2ELi2ELb0E": (9, 9),
         "latent_attention_kernelILi1ELi4ELb1E": (5, 5), "latent_attention_kernelILi2ELi2ELb1E": (5, 5),
         "heads_ring_kernelILi4E": (1, 2), "heads_ring_kernelILi8E": (2, 4),
         "heads_ring_kernelILi12E": (3, 6), "heads_ring_kernelILi16E": (4, 8)}


@pytest.mark.parametrize("kernel", RINGS)
def test_ring_waits_count_a_steps_loads(functions, kernel):
    (code,) = [c for name, c in functions.items() if kernel in name]
    loads, wait = RINGS[kernel]
    waits = ring_waits(code, wait)
    assert waits, "no wait of this count"
    for w in waits:
        least = least_loads(code, w, waits)
        assert least is None or least >= loads, f"{least} loads from the wait at {code[w][3]:#x}"
    assert any(least_loads(code, w, waits) == loads for w in waits)
    assert least_loads(code, -1, waits) >= 3 * loads  # before the first step: of all slots of the ring but one
    assert not any(name.startswith("scratch_") for name, *_ in code)


def test_the_loads_of_a_path_are_counted():
    wait = "s_waitcnt vmcnt(2) lgkmcnt(0)"
    code = _code(wait, "s_barrier", LOAD, ("s_cbranch_scc0 2", 20), LOAD, ("s_cbranch_scc1 65530", 0), "s_endpgm")
    assert ring_waits(code, 2) == {0}
    assert least_loads(code, 0, {0}) == 1  # round the second
    assert least_loads(code, -1, {0}) == 0
    assert least_loads(code, 0, {99}) is None


def _code(*lines):
    return parse([(4 * i, text, target) for i, (text, target) in enumerate((l, None) if isinstance(l, str) else l for l in lines)])


LOAD = "buffer_load_dwordx4 v1, s[8:11], 0 offen lds"


def test_the_check_finds_what_it_looks_for():
    read = "v_readlane_b32 s10, v3, s2"
    assert len(hazards(_code(read, "s_add_u32 m0, s4, 16", "s_nop 0", LOAD))) == 1  # two states
    assert len(hazards(_code(read, "s_nop 3", LOAD))) == 1
    assert hazards(_code(read, "s_nop 4", LOAD)) == []
    assert hazards(_code(read, "s_add_u32 m0, s4, 16", "s_nop 3", LOAD)) == []
    assert hazards(_code("s_mov_b32 s10, s2", "s_nop 0", LOAD)) == []           # a scalar instruction's result is waited for
    assert hazards(_code("v_readlane_b32 s12, v3, s2", LOAD)) == []               # another register
    assert len(hazards(_code("v_cmp_gt_u32_e64 s[8:9], v0, v1", LOAD))) == 1
    assert len(hazards(_code("s_add_u32 m0, s4, 16", LOAD))) == 1
    # around a branch: the write stands at the end of a loop whose head loads
    loop = _code("s_nop 7", LOAD, "s_nop 4", read, ("s_cbranch_scc1 65531", 4), "s_endpgm")
    assert len(hazards(loop)) == 1
    assert hazards(_code("s_nop 7", LOAD, read, "s_nop 4", ("s_cbranch_scc1 65531", 4), "s_endpgm")) == []
    # m0
    assert others_with_m0(_code("s_add_u32 m0, s4, 16", "s_nop 3", LOAD)) == []
    assert len(others_with_m0(_code("s_add_u32 m0, s4, 16", "s_nop 3", LOAD, LOAD))) == 1
    assert len(others_with_m0(_code("s_mov_b32 m0, s4", "s_nop 3", LOAD))) == 2
