"""The form of the kernels' 16-byte buffer stores, read from their sources.

The data of a store of more than 8 bytes must not be written anew by the next
instruction.  The compiler leaves a wait state there only where the store has
no scalar offset, so each gives its whole offset in the lanes' register.
"""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_105_amd", "csrc")


def arguments(text, at):
    """The arguments of the call whose opening bracket is at text[at]."""
    depth, out, start = 0, [], at + 1
    for i in range(at, len(text)):
        depth += text[i] in "([{"
        depth -= text[i] in ")]}"
        if depth == 1 and text[i] == "," or depth == 0:
            out.append(text[start:i].strip())
            start = i + 1
        if depth == 0:
            return out
    raise AssertionError("unbalanced call")


def test_wide_buffer_stores_have_no_scalar_offset():
    found = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        with open(path) as f:
            text = f.read()
        for m in re.finditer(r"raw_buffer_store_b(96|128)\(", text):
            args = arguments(text, m.end() - 1)
            line = text.count("\n", 0, m.start()) + 1
            assert len(args) == 5 and args[3] == "0", f"{os.path.basename(path)}:{line}: {args}"
            found += 1
    assert found >= 3
