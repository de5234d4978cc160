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


def test_states_that_may_be_one_buffer_are_not_restrict():
    """la.h lets S be S0, dS0 be dS, y be x and dx be dy or x."""
    for name, params in (("gated_delta.cu", r"(const float|float)\* __restrict__ (S0|S_out|dS0)\b|const float\* __restrict__ dS\b"),
                         ("tc_gated_delta_states.cuh", r"__restrict__ (S0|S_out)\b"),
                         ("tc_gated_delta_bwd.cu", r"__restrict__ (segdS|dS0|S0)\b"),
                         ("layer_norm.cu", r"__restrict__ (x|y|dx|dy)\b")):
        assert not re.search(params, code(text(name))), name


def file_tag(name):
    """dbg::file_tag in la_internal.cuh: FNV-1a of the base name, folded to 16 bits."""
    h = 2166136261
    for c in name.encode():
        h = (h ^ c) * 16777619 & 0xFFFFFFFF
    return (h ^ h >> 16) & 0xFFFF


def test_a_failed_index_check_names_its_file():
    """The debug build reports a check's site by a tag of its file: every source is in the list that names it, no two alike."""
    listed = re.search(r"kFiles\[\] = \{(.*?)\}", text("api.cu"), re.S).group(1)
    assert sorted(re.findall(r'"([^"]+)"', listed)) == FILES
    assert len({file_tag(n) for n in FILES}) == len(FILES)
