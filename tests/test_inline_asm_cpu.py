"""Inline assembly says what it overwrites: a statement that writes m0 lists it as clobbered, so that the compiler keeps
nothing there across it."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int8_dequant_dot_amd", "csrc")


def statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        if os.path.isfile(path):
            with open(path) as f:
                for m in re.finditer(r"\basm(?:\s+volatile)?\s*\((.*?)\);", f.read(), re.S):
                    yield os.path.basename(path), m.group(1)


def test_m0_is_clobbered_where_it_is_written():
    writers = [(name, text) for name, text in statements() if re.search(r"\bs_\w+\s+m0\s*,", text)]
    assert writers
    for name, text in writers:
        clobbers = text.rsplit(":", 1)[1]
        assert '"m0"' in clobbers, (name, text)
