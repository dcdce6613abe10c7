"""Reads of a matrix instruction's result that come too soon, over all paths
through a listing of gfx950 code.

A matrix instruction writes its result some passes of four cycles after it was
issued, and nothing holds back a later instruction that reads it, but another
matrix instruction that takes it as its own C: the program has to leave that
many wait states between, of which every instruction is one and `s_nop n` is n
+ 1.  The compiler does, but has been seen not to where a branch lay between.
"""
import re

# Wait states between a matrix instruction and a read of its result by another
# kind of instruction, or as a factor: its passes and four (two for the one that
# multiplies float32), which the compiler keeps to in straight code for gfx950.
WAITS = {"v_mfma_f32_16x16x32_bf16": 4 + 4, "v_mfma_f32_32x32x16_bf16": 8 + 4, "v_mfma_f32_16x16x4_f32": 8 + 2}
# And between a vector instruction that writes scalar registers and a memory instruction that reads them.
SCALAR = 5
_REGISTERS = re.compile(r"(?<![\w.])([av])(?:\[(\d+):(\d+)\]|(\d+)(?!\w))")
_SCALARS = re.compile(r"(?<![\w.])s(?:\[(\d+):(\d+)\]|(\d+)(?!\w))")
_LINE = re.compile(r"^\t(\S.*?)\s*// ([0-9A-F]+):.*?(?:<\S+?(?:\+0x([0-9a-f]+))?>)?$")


def registers(text):
    return {(m[1], k) for m in _REGISTERS.finditer(text) for k in range(int(m[2] or m[4]), int(m[3] or m[4]) + 1)}


def functions(listing):
    """(name, [(instruction, index that it branches to or None)]) of llvm-objdump's listing."""
    for part in re.split(r"^(?=[0-9a-f]{16} <)", listing, flags=re.M)[1:]:
        head, _, body = part.partition("\n")
        lines = [m for m in map(_LINE.match, body.split("\n")) if m]
        if not lines:
            continue
        start = int(head[:16], 16)
        index = {int(m[2], 16): n for n, m in enumerate(lines)}
        code = []
        for m in lines:
            branches = m[1].startswith(("s_branch", "s_cbranch"))
            code.append((m[1], index[start + int(m[3] or "0", 16)] if branches else None))
        yield head[18:-2], code


def scalars(text):
    return {k for m in _SCALARS.finditer(text) for k in range(int(m[1] or m[3]), int(m[2] or m[3]) + 1)}


def _walk(code, n, need, stops):
    """Goes on from instruction n over all paths until `stops(instruction, operands)` or `need` wait states; yields what
    `stops` calls a read, with the wait states before it."""
    def after(k):
        text, target = code[k]
        if text.startswith(("s_endpgm", "s_branch")):
            return [] if target is None else [target]
        return [x for x in (k + 1, target) if x is not None and x < len(code)]

    seen, todo = {}, [(k, 0) for k in after(n)]
    while todo:
        at, states = todo.pop()
        if states >= need or seen.get(at, need) <= states:
            continue
        seen[at] = states
        op, _, args = code[at][0].partition(" ")
        what = stops(op, args)
        if what == "read":
            yield code[at][0], states
        elif what is None:
            todo += [(k, states + (int(args) + 1 if op == "s_nop" else 1)) for k in after(at)]


def too_soon(code):
    """(writer, reader, wait states between) of one function."""
    found = set()
    for n, (text, _) in enumerate(code):
        op, _, rest = text.partition(" ")
        if op.startswith("v_mfma"):
            result = registers(rest.split(",")[0])

            def stops(other, args):
                if other.startswith("v_mfma"):
                    d, a, b = args.split(", ")[:3]
                    if (registers(a) | registers(b)) & result:
                        return "read"
                    return "over" if registers(d) & result else None   # adds to it, or takes its place, in order
                return "read" if other[0] != "s" and registers(args) & result else None

            found |= {(text, *read) for read in _walk(code, n, WAITS[op], stops)}
        elif op.startswith(("v_readfirstlane", "v_readlane", "v_cmp")) and scalars(rest.split(",")[0]):
            written = scalars(rest.split(",")[0])

            def stops(other, args):
                if other.startswith(("global_", "buffer_", "flat_", "scratch_")):
                    return "read" if scalars(args) & written else None
                writes = other[0] == "s" and not other.startswith(("s_cmp", "s_bit", "s_cbranch", "s_wait", "s_nop"))
                return "over" if writes and scalars(args.split(",")[0]) >= written else None

            found |= {(text, *read) for read in _walk(code, n, SCALAR, stops)}
    return found
