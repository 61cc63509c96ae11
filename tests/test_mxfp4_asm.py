"""CPU check of the assembly of the products by expert on microscaled FP4 rows.  The kernel of the
largest tiles writes its matrix instructions out (their accumulators stay in place that way), and
the compiler does not know the waits that those need: no vector instruction may write an operand of
one less than two wait states before it, none may read its result less than eight behind it (a
4-pass instruction's result takes seven), and no loads through flat addresses may stand between
the loads that the kernels count."""

import re
import subprocess

import pytest

from routed_moe_layer_amd import build as b

OPERAND, RESULT = 2, 8


def _registers(token, kind):
    m = re.match(rf"{kind}\[(\d+):(\d+)\]$", token)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.match(rf"{kind}(\d+)$", token)
    return {int(m.group(1))} if m else set()


def _kernels(text):
    """{kernel name: [(opcode, operands, whether it is written out)]}"""
    found, code, written = {}, None, False
    for line in text.splitlines():
        m = re.match(r"(_ZN4rmoe\w+):", line)
        if m:
            code = found.setdefault(m.group(1), [])
        if "#ASMSTART" in line or "#ASMEND" in line:
            written = "#ASMSTART" in line
        body = line.split(";")[0].strip()
        if code is None or not body or body.endswith(":") or body.startswith("."):
            continue
        op, _, rest = body.partition(" ")
        code.append((op, [a.strip().split(" ")[0] for a in rest.split(",")], written))
    return found


def hazards(code):
    """Where a written-out matrix instruction's waits are missing."""
    bad, states = [], 0
    wrote, results = {}, {}              # VGPR: when a vector instruction wrote it; AGPR: its product
    for i, (op, args, written) in enumerate(code):
        mfma = op.startswith("v_mfma")
        if mfma and written:
            for r in set().union(*(_registers(a, "v") for a in args[1:])):
                if states - wrote.get(r, -99) < OPERAND:
                    bad.append((i, op, f"v{r} written {states - wrote[r]} wait states before"))
        elif op.startswith(("v_", "ds_", "global_", "buffer_", "scratch_")) and not mfma:
            for r in set().union(*(_registers(a, "a") for a in args)):
                if states - results.get(r, -99) < RESULT:
                    bad.append((i, op, f"a{r} read {states - results[r]} wait states behind its product"))
        states += int(args[0]) + 1 if op == "s_nop" else 1
        if mfma and written:
            for r in _registers(args[0], "a"):
                results[r] = states
        elif op.startswith("v_"):
            for r in _registers(args[0], "v"):
                wrote[r] = states
    return bad


def test_the_check_sees_what_it_looks_for():
    mfma = ("v_mfma_scale_f32_16x16x128_f8f6f4", ["a[0:3]", "v[0:3]", "v[4:7]", "a[0:3]", "v8", "v9"], True)
    write, nop = ("v_mov_b32_e32", ["v5", "v20"], False), lambda n: ("s_nop", [str(n)], False)
    read = ("v_accvgpr_read_b32", ["v30", "a2"], False)
    assert hazards([write, mfma]) and hazards([write, nop(0), mfma]) and not hazards([write, nop(1), mfma])
    assert hazards([mfma, read]) and hazards([mfma, nop(6), read]) and not hazards([mfma, nop(7), read])


def _assembly(name):
    r = subprocess.run([b.HIPCC, *b.COMMON_FLAGS, "--cuda-device-only", "-S", f"{b.CSRC}/{name}", "-o", "-"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return _kernels(r.stdout)


@pytest.mark.slow
def test_the_written_out_products_have_their_waits():
    kernels = {n: c for n, c in _assembly("grouped_mxfp4_big.hip").items() if "kernel" in n}
    assert len(kernels) == 2
    for name, code in kernels.items():
        assert sum(op.startswith("v_mfma") and w for op, _, w in code) >= 480
        assert not hazards(code), (name, hazards(code)[:5])
        assert not any(op.startswith(("flat_load", "flat_store")) for op, _, _ in code), name
