"""Operands that a kernel's own result may overwrite, read by ordinary loads: the non-coherent path
(ld.global.nc, __ldg) is for memory that does not change while a kernel runs, and such a load need
not stay before the store to its address. What a schedule makes of it does not show in results,
so this is checked in the source text; the results in place are tested on the GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mxfp8_block_scaled_05_gb300", "csrc")
NON_COHERENT = r"ld_nc\w*|__ldg|load_once"


def body(file, name):
    """The text of a __global__ function or a device helper, without comments."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())
    m = re.search(r"\b" + name + r"\([^;{]*\)\s*\{(.*?)\n\}", text, re.S)
    assert m, name
    return m[1]


def reads(text, how):
    """First arguments of the calls of `how` in the text."""
    return re.findall(r"\b(?:" + how + r")(?:<[^>]*>)?\(([^,)]*)", text)


def test_rows_gradient_in_place_of_the_rows():
    kernel = body("routing.cu", "combine_grad_kernel")
    assert [a for a in reads(kernel, "load_operand<kRows>") if a.startswith("y ")]
    assert not [a for a in reads(kernel, NON_COHERENT) if re.match(r"y\b", a)]
    helper = body("routing.cu", "load_operand")
    assert re.search(r"if constexpr \(kMayBeWritten\) return \*p;", helper)


def test_activation_in_place_of_its_gradient():
    kernel = body("swiglu.cu", "swiglu_grad_kernel")
    again = re.search(r"if constexpr \(kAgain\) \{(.*?)\} else \{(.*?)\}", kernel, re.S)
    assert again and reads(again[1], "load16_operand") == ["p.grad + q.row * p.width + q.c"]
    rest = kernel.replace(again[0], "")   # nor is it read anywhere else
    assert "p.grad " not in rest and "p.grad," not in rest
    helper = body("swiglu.cu", "load16_operand")
    assert not re.search(NON_COHERENT, helper) and ".nc" not in helper
    assert '"memory"' in helper           # no store moves before it
