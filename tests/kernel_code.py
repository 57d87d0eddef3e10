"""The device code of a source file as LLVM IR, compiled with the library's own
flags, for checks of what no run can show: which lanes are active where a
register is read by others, and what orders LDS accesses of different lanes."""
import os
import re
import subprocess

from fsdp_sharded_optimizer_step_amd import build_ext

HIPCC, OPT = "/opt/rocm/bin/hipcc", "/opt/rocm/llvm/bin/opt"


def available():
    return os.path.exists(HIPCC) and os.path.exists(OPT)


def compile_ir(source, folder):
    """Path of the optimised IR of csrc/<source>."""
    out = os.path.join(str(folder), source + ".ll")
    flags = [f for f in build_ext.FLAGS if f not in ("-fPIC", "-shared", "-Wall")]
    subprocess.run([HIPCC, *flags, "--cuda-device-only", "-S", "-emit-llvm",
                    os.path.join(build_ext.CSRC, source), "-o", out],
                   check=True, stderr=subprocess.DEVNULL)
    return out


class Block:
    def __init__(self):
        self.lines, self.next, self.divergent = [], [], False


def functions(ir, keep):
    """{name: {label: Block}} of the functions whose name holds one of `keep`,
    from the compiler's uniformity analysis: a block's instructions, its
    successors, and whether lanes part at its end.  The first block is the
    entry."""
    text = subprocess.run([OPT, "-disable-output", "-passes=print<uniformity>", ir],
                          check=True, capture_output=True, text=True)
    found, blocks, block = {}, None, None
    for line in (text.stdout + text.stderr).splitlines():
        if line.startswith("UniformityInfo for function"):
            name = line.split("'")[1]
            blocks = found.setdefault(name, {}) if any(k in name for k in keep) else None
        if blocks is None:
            continue
        if line.startswith("BLOCK "):
            block = blocks[line.split()[1]] = Block()
        elif block is not None and line.startswith("END BLOCK"):
            block = None
        elif block is not None and line.strip() not in ("DEFINITIONS", "TERMINATORS"):
            parted = line.lstrip().startswith("DIVERGENT:")
            code = line.replace("DIVERGENT:", "").strip()
            block.lines.append(code)
            if re.match(r"(br|switch|ret|unreachable)\b", code):
                block.next = re.findall(r"label %([\w.]+)", code)
                block.divergent = parted and len(set(block.next)) > 1
    return found


def post_dominators(blocks):
    """{label: labels that every path from it to the end passes, itself among
    them}."""
    every = set(blocks)
    pd = {b: ({b} if not blocks[b].next else set(every)) for b in blocks}
    changed = True
    while changed:
        changed = False
        for b in reversed(list(blocks)):
            if blocks[b].next:
                new = {b} | set.intersection(*(pd[s] for s in blocks[b].next))
                if new != pd[b]:
                    pd[b], changed = new, True
    return pd


def parted(blocks):
    """Labels of the blocks that some lanes of a wave may pass without the
    others: those between a divergent branch and the first block that all its
    paths come to."""
    pd, out = post_dominators(blocks), set()
    for b, block in blocks.items():
        if not block.divergent:
            continue
        todo = [s for s in block.next if s not in pd[b] - {b}]
        seen = set()
        while todo:
            x = todo.pop()
            if x in seen:
                continue
            seen.add(x)
            todo += [s for s in blocks[x].next if s not in pd[b] - {b}]
        out |= seen
    return out


def instructions(ir, keep):
    """The same from the IR alone, without the analysis, which takes minutes on
    kernels of many unrolled instructions."""
    found, blocks, block = {}, None, None
    with open(ir) as f:
        for line in f:
            if line.startswith("define "):
                name = re.search(r"@([\w.]+)\(", line).group(1)
                blocks = block = None
                if any(k in name for k in keep):
                    blocks = found[name] = {}
                    block = blocks[""] = Block()
            elif blocks is None:
                continue
            elif line.startswith("}"):
                blocks = None
            elif re.match(r"[\w.]+:", line):
                block = blocks[line.split(":")[0]] = Block()
            elif line.strip():
                block.lines.append(line.strip())
                # a switch's targets stand in lines of their own
                block.next += re.findall(r"label %([\w.]+)", line)
    return found
