"""Finds, in the assembly of kernels built here, results of matrix instructions
that another pipe reads or writes before they are there.

The hardware does not hold such an instruction back: the program has to leave
passes + 3 wait states (one for each instruction, n + 1 for s_nop n) between a
matrix instruction and any other use of its result, whichever way control goes."""
import re

# passes of the instructions that the row operators use (scaled ones: with 8-bit operands, with two 4-bit ones)
PASSES = {"v_mfma_scale_f32_32x32x64_f8f6f4": (16, 8), "v_mfma_scale_f32_16x16x128_f8f6f4": (8, 4),
          "v_mfma_f32_32x32x16_bf16": (8, 8), "v_mfma_f32_16x16x32_bf16": (4, 4)}


def registers(text):
    out = set()
    for kind, first, last in re.findall(r"\b([va])\[(\d+):(\d+)\]", text):
        out |= {(kind, i) for i in range(int(first), int(last) + 1)}
    return out | {(kind, int(i)) for kind, i in re.findall(r"(?<![\w\[:])([va])(\d+)\b", text)}


def functions(asm):
    """{name: [label or instruction, ...]}; labels end with a colon."""
    out, code = {}, None
    for line in asm.splitlines():
        line = line.split(";")[0].strip()
        if re.match(r"_Z\w+:$", line):
            code = out[line[:-1]] = []
        elif code is not None and line and (not line.startswith(".") or re.match(r"\.L\w+:$", line)):
            code.append(line)
    return out


def needed(ins):
    name = ins.split()[0]
    if name not in PASSES:
        raise ValueError(f"{name}: passes not known")
    return PASSES[name]["cbsz:4 blgp:4" in ins] + 3


def early_uses(code):
    """(matrix instruction, its user, wait states between, needed) in one function."""
    at = {line[:-1]: i for i, line in enumerate(code) if line.endswith(":")}
    found = []
    for i, ins in enumerate(code):
        if not ins.startswith("v_mfma"):
            continue
        need, dst = needed(ins), registers(ins.split(None, 1)[1].split(",")[0])
        paths, seen = [(i + 1, 0)], {}
        while paths:
            j, waits = paths.pop()
            while j < len(code) and waits < need:
                line = code[j]
                if line.endswith(":"):
                    if seen.get(j, need) <= waits:
                        break
                    seen[j] = waits
                    j += 1
                    continue
                name, _, args = line.partition(" ")
                if name == "s_nop":
                    waits += int(args, 0)
                elif name == "s_branch":
                    j = at[args.strip()] - 1
                elif name.startswith("s_cbranch"):
                    paths.append((at[args.strip()], waits + 1))
                elif name == "s_endpgm":
                    break
                elif name.startswith("v_mfma"):
                    out, a, b = re.split(r",\s*(?![^\[]*\])", args)[:3]
                    if registers(out) == dst and not (registers(a) | registers(b)) & dst:
                        break  # accumulates: the hardware chains these
                    if registers(args) & dst:
                        found.append((ins, line, waits, need))
                        break
                elif registers(args) & dst:
                    found.append((ins, line, waits, need))
                    break
                waits += 1
                j += 1
    return found
