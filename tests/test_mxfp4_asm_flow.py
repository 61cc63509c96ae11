"""CPU check of the assembly of the 256 x 256 tiles' written-out matrix instructions along every path
through the kernel, over branches and back edges: between a vector instruction and a product that
reads what it wrote, operands, scales or the accumulator that stays in place, lie two wait states;
between a product and any other instruction that reads or overwrites its result lie eight, which is
what gfx950 takes for these (4 passes) and what its compiler puts behind the same instruction's
builtin.  That rule is looked up by compiling the builtin, not taken from here."""

import functools
import re
import subprocess

import pytest

from routed_moe_layer_amd import build as b

OPERAND, RESULT = 2, 8


def _registers(token, kinds="va"):
    """{"v0", "a5", ...} of an operand."""
    m = re.match(rf"([{kinds}])\[(\d+):(\d+)\]$", token)
    if m:
        return {f"{m.group(1)}{i}" for i in range(int(m.group(2)), int(m.group(3)) + 1)}
    m = re.match(rf"([{kinds}])(\d+)$", token)
    return {token} if m else set()


def kernels(text):
    """{kernel name: lines}, a line a label (text) or an instruction (opcode, operands, whether it
    is written out)."""
    found, code, written = {}, None, False
    for line in text.splitlines():
        m = re.match(r"(_ZN4rmoe\w+kernel\w+):", line)
        if m:
            code = found.setdefault(m.group(1), [])
        if "#ASMSTART" in line or "#ASMEND" in line:
            written = "#ASMSTART" in line
        body = line.split(";")[0].strip()
        if code is None or not body:
            continue
        if body.endswith(":"):
            if body.startswith(".LBB"):
                code.append(body[:-1])
            continue
        if body.startswith("."):
            if body.startswith(".end_amdhsa_kernel") or body.startswith(".section"):
                code = None
            continue
        op, _, rest = body.partition(" ")
        code.append((op, [t for a in rest.split(",") for t in a.strip().split(" ")[:1]], written))
    return found


def _blocks(code):
    """([instructions], [successors]) of each basic block, the first one the entry."""
    starts, labels, out = [0], {}, []
    for line in code:
        if isinstance(line, str):
            if out and len(out) != starts[-1]:
                starts.append(len(out))
            labels[line] = len(starts) - 1
        else:
            out.append(line)
            if line[0].startswith(("s_cbranch", "s_branch", "s_endpgm", "s_setpc")):
                starts.append(len(out))
    blocks = []
    for i, at in enumerate(starts):
        end = starts[i + 1] if i + 1 < len(starts) else len(out)
        ins = out[at:end]
        last = ins[-1][0] if ins else ""
        to = [labels[ins[-1][1][0]]] if last.startswith(("s_cbranch", "s_branch")) else []
        if not last.startswith(("s_branch", "s_endpgm", "s_setpc")) and i + 1 < len(starts):
            to.append(i + 1)
        blocks.append((ins, to))
    return blocks


def _step(state, ins, bad):
    """The state behind an instruction: by register, wait states since a vector instruction wrote
    it ("w") or a written-out product did ("p"), as far as that is still too few."""
    op, args, written = ins
    product = op.startswith("v_mfma") and written
    if bad is not None:
        if product:
            for r in set().union(*(_registers(a) for a in args)):
                if state.get(("w", r), OPERAND) < OPERAND:
                    bad.append(f"{op} {','.join(args)}: {r} written {state['w', r]} wait states before")
        elif op.startswith(("v_", "ds_", "global_", "buffer_", "scratch_", "flat_")):
            # (products by the builtin read and write results as any other instruction would)
            for r in set().union(*(_registers(a, "a") for a in args)):
                if state.get(("p", r), RESULT) < RESULT:
                    bad.append(f"{op} {','.join(args)}: {state['p', r]} wait states behind the product in {r}")
    n = int(args[0]) + 1 if op == "s_nop" else 1
    limit = {"w": OPERAND, "p": RESULT}
    state = {k: v + n for k, v in state.items() if v + n < limit[k[0]]}
    if product:
        state.update({("p", r): 0 for r in _registers(args[0], "a")})
    elif op.startswith("v_"):
        state.update({("w", r): 0 for r in _registers(args[0])})
    return state


def hazards(code):
    """Where a path leads to a written-out product or away from one without its waits."""
    blocks = _blocks(code)
    entry, queue = {0: {}}, [0]
    while queue:
        i = queue.pop()
        state = entry[i]
        for ins in blocks[i][0]:
            state = _step(state, ins, None)
        for j in blocks[i][1]:
            old = entry.get(j)
            new = state if old is None else {k: min(old.get(k, 99), state.get(k, 99))
                                             for k in old.keys() | state.keys()}
            if new != old:
                entry[j] = new
                queue.append(j)
    bad = []
    for i, state in entry.items():
        for ins in blocks[i][0]:
            state = _step(state, ins, bad)
    return bad


@functools.lru_cache(maxsize=None)
def _text(source):
    r = subprocess.run([b.HIPCC, *b.COMMON_FLAGS, "--cuda-device-only", "-S", source, "-o", "-"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


def _assembly(source):
    return kernels(_text(source))


def scratch(text):
    """{kernel name: bytes of scratch a lane}"""
    return {m.group(1): int(m.group(2)) for m in re.finditer(
        r"\.amdhsa_kernel (\w+).*?\.amdhsa_private_segment_fixed_size (\d+)", text, re.S)}


MFMA = ("v_mfma_scale_f32_16x16x128_f8f6f4", ["a[0:3]", "v[0:3]", "v[4:7]", "a[0:3]", "v8", "v9"], True)
READ, OTHER = ("v_accvgpr_read_b32", ["v30", "a2"], False), ("s_add_u32", ["s0", "s0", "1"], False)
LOOP, AGAIN, END = ".LBB0_1", ("s_cbranch_scc1", [".LBB0_1"], False), ("s_endpgm", [""], False)


def _nop(n):
    return ("s_nop", [str(n)], False)


@pytest.mark.parametrize("write", ["v5", "v8", "a1", "v[2:3]"])
def test_sees_operands_scales_and_accumulators_written_just_before(write):
    w = ("v_mov_b32_e32", [write, "v20"], False)
    assert hazards([w, MFMA, END]) and hazards([w, _nop(0), MFMA, END])
    assert not hazards([w, _nop(1), MFMA, END]) and not hazards([w, OTHER, OTHER, MFMA, END])


def test_sees_results_read_or_overwritten_too_early():
    clear = ("v_accvgpr_write_b32", ["a2", "0"], False)
    for use in (READ, clear):
        assert hazards([MFMA, use, END]) and hazards([MFMA, _nop(6), use, END])
        assert not hazards([MFMA, _nop(7), use, END])


def test_sees_what_a_back_edge_and_a_jump_bring_together():
    # the loop's end meets its head: the product is in no straight line in front of the reader
    assert hazards([LOOP, READ, _nop(7), MFMA, AGAIN, END])
    assert not hazards([LOOP, READ, _nop(1), MFMA, _nop(7), AGAIN, END])
    write = ("v_mov_b32_e32", ["v5", "v20"], False)
    assert hazards([_nop(1), LOOP, MFMA, _nop(7), write, AGAIN, END])
    # a jump over the wait
    skip = ("s_cbranch_execz", [".LBB0_2"], False)
    assert hazards([MFMA, skip, _nop(7), ".LBB0_2", READ, END])
    # and what no path joins is none
    assert not hazards([MFMA, ("s_branch", [".LBB0_2"], False), LOOP, READ, END, ".LBB0_2", _nop(7), END])


@pytest.mark.slow
def test_the_compiler_puts_as_many_wait_states_behind_the_builtin(tmp_path):
    source = tmp_path / "one.hip"
    source.write_text("""
#include "grouped_mxfp4.h"
namespace rmoe {
__global__ void one_kernel(const u32x4* x, f32x4* out, uint32_t s) {
  const f32x4 r = mx_mma<0>(x[threadIdx.x], x[64 + threadIdx.x], f32x4{0, 0, 0, 0}, s, s);
  out[threadIdx.x] = r;
}
}
""")
    code = next(iter(_assembly(str(source)).values()))
    at = next(i for i, line in enumerate(code) if line[0].startswith("v_mfma"))
    dest, states = _registers(code[at][1][0]), 0
    for op, args, _ in code[at + 1:]:
        if any(dest & _registers(a) for a in args):
            break
        states += int(args[0]) + 1 if op == "s_nop" else 1
    assert states == RESULT


@pytest.mark.slow
def test_the_written_out_products_have_their_waits_on_every_path():
    found = _assembly(f"{b.CSRC}/grouped_mxfp4_big.hip")
    assert len(found) == 2
    for name, code in found.items():
        n = sum(not isinstance(i, str) and i[0].startswith("v_mfma") and i[2] for i in code)
        assert n >= 480
        assert sum(len(to) for _, to in _blocks(code)) > 40
        assert not hazards(code), (name, hazards(code)[:5])


@pytest.mark.slow
def test_only_the_activation_spills_and_no_more_than_is_known():
    """33 registers of the large tiles with the activation; the plain ones none."""
    found = scratch(_text(f"{b.CSRC}/grouped_mxfp4_big.hip"))
    assert len(found) == 2
    for name, size in found.items():
        assert size <= (136 if "ILb1E" in name else 0), name
