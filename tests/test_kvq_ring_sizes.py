"""The rings that the barrier model of the quantised-cache decode kernel runs are the kernel's: worked out here from the constants
and formulas in its source, for every head size, block size and number of bits."""
import math
import os
import re

import test_kvq_ring_model as model

SOURCE = os.path.join(os.path.dirname(__file__), "..", "bit_grouped_expert_top_gb300", "csrc", "kvq_decode.cu")
with open(SOURCE) as _f:
    TEXT = re.sub(r"//[^\n]*", "", _f.read())


def _expr(c: str) -> str:
    """A C expression of integers as Python: / is the whole division, a ? b : c the conditional."""
    choice = re.compile(r"((?:\w+\([^()]*\)|[^()?:])+)\?([^()?:]+):([^()?:]+)")
    return choice.sub(r"(\2 if \1 else \3)", c).replace("/", "//").strip()


def _constants():
    names = {}
    for name, value in re.findall(r"constexpr int (k\w+) = ([^;]+);", TEXT):
        if "sizeof" not in value:
            try:
                names[name] = eval(_expr(value), {}, {**names, **_functions(names)})
            except (NameError, SyntaxError):
                pass   # several names in a line, or a constant of a template's parameters
    return names


def _functions(names):
    got = {}
    for name, args, body in re.findall(r"constexpr (?:int|bool) (\w+)\(([^)]*)\)\s*\{([^}]*)\}", TEXT):
        params = [a.split()[-1] for a in args.split(",")]
        got[name] = _function(params, body, names, got)
    return got


def _function(params, body, names, functions):
    def call(*values):
        scope = {**names, **functions, **dict(zip(params, values))}
        for what, value in re.findall(r"(?:const int (\w+) =|return) ([^;]+);", body):
            result = eval(_expr(value), {}, scope)
            if not what:
                return result
            scope[what] = result
    return call


def _size_of_fixed(names) -> int:
    """sizeof(Fixed), of the product's build."""
    body = re.search(r"struct Fixed \{(.*?)\n\};", TEXT, re.S)[1]
    body = re.sub(r"#ifdef.*?#endif", "", body, flags=re.S)
    size = 0
    for align, kind, fields in re.findall(r"(?:alignas\((\d+)\) )?(uint64_t|int|float) ([^;]+);", body):
        width = {"uint64_t": 8, "int": 4, "float": 4}[kind]
        step = max(width, int(align or 1))
        size = (size + step - 1) // step * step
        for field in fields.split(","):
            size += width * math.prod(eval(_expr(n), {}, names) for n in re.findall(r"\[([^\]]+)\]", field))
    return (size + 7) // 8 * 8


def test_the_model_runs_the_rings_of_the_kernel():
    names = _constants()
    assert names["kNW"] == model.WARPS and names["kMaxStages"] > 1
    fixed = _size_of_fixed(names)
    assert re.search(r"constexpr int kFixed = \(sizeof\(Fixed\) \+ 127\) / 128 \* 128;", TEXT)
    names["kFixed"] = (fixed + 127) // 128 * 128
    functions = _functions(names)
    rings = set()
    for D in (64, 128, 256):
        for bs in (32, 64, 128):
            for bits in (4, 8):
                rings.add((functions["stages_for"](D, bs, bits), bs // functions["unit_of"](D)))
    assert rings == set(model.RINGS)
