"""Rules that every kernel source keeps, read off the sources."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "causal_linear_attention_phi_gb300", "csrc")
FILES = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu*")))


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def functions(src):
    """The top-level pieces of a source, each up to a closing brace in the first column."""
    return [p for p in re.split(r"^}.*$", src, flags=re.M) if p.strip()]


def code(src):
    return re.sub(r"//[^\n]*", "", src)


# The armed copies of a buffer (or those a block may have issued) are waited for on the way out.
LEAVES_NONE = re.compile(r"if \(\w*armed\w*(\[\w+\])? >= 0\) mbar_wait\(|drain\(|if \(!ok\) mbar_wait\(")


@pytest.mark.parametrize("name", FILES)
def test_no_block_leaves_copies_in_flight(name):
    """A function that arms a barrier for copies waits, after its last one, for what a wait that ran out left in flight."""
    for piece in functions(text(name)):
        body = code(piece)
        armed = [m.end() for m in re.finditer(r"\bmbar_arrive_expect_tx\(&?\w", body)
                 if "void mbar_arrive_expect_tx" not in body[m.start() - 5:m.end()]]
        if not armed:
            continue
        where = re.findall(r"\b(\w+)\([^;{]*\{", body)
        waits = [m.start() for m in LEAVES_NONE.finditer(body)]
        assert waits and max(waits) > max(armed), "%s: %s arms copies and leaves none waited for" % (name, where[:1])


def test_the_rule_sees_every_file_that_copies():
    copying = {n for n in FILES if re.search(r"\bmbar_arrive_expect_tx\(", code(text(n)))} - {"sm100.cuh"}
    seen = {n for n in copying if any(LEAVES_NONE.search(code(p)) for p in functions(text(n)))}
    assert copying == seen and len(copying) >= 8
