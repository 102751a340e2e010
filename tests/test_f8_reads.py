"""How the weighted sum reads what it may also write, by the kernel's source: the values of a
run cannot show it."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "any_precision_weight_gb300",
                      "csrc", "pw_f8_rows.cu")


def test_a_residual_that_may_be_the_output_is_read_by_ordinary_loads():
    """The read-only path (__ldg) is defined for memory that the kernel does not write."""
    text = re.sub(r"//.*", "", open(SOURCE).read())
    reads = re.findall(r"load_cols<([^>]*)>\(static_cast<const (\w)\*>\(p\.(\w+)\)", text)
    assert {(t, name) for _, t, name in reads} == {("O", "res"), ("Y", "y")}
    for args, _, name in reads:
        assert args.split(", ")[2:] == ["true" if name == "res" else "false"], (name, args)
    body = re.search(r"load_cols\(const T\* row.*?\n}\n", text, re.S).group(0)
    assert re.findall(r"\S+ : __ldg\(", body) == ["*from : __ldg("] and "OUT ? *from" in body
    assert "__ldg(p.res" not in text
