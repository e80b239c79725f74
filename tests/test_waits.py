"""A wait that ran out is not forgotten: what the warps that feed the chunk kernel do about it, read
in its source (no wait is made to run out on a GPU for it)."""
import os
import re

import ternary_weight_ptq1_gb300 as P


def _feeding():
    with open(os.path.join(P._build.CSRC, "k_attn_chunk.cu")) as f:
        text = f.read()
    text = text[text.index("K and V tiles through the ring"):]
    text = re.sub(r"//[^\n]*", "", text[:text.index("copies_but<0>();")])
    return re.sub(r"\s+", " ", text)


def test_a_wait_that_ran_out_stays_known():
    """These warps go on with a batch of copies before they agree on `ok`, so a new value has the old one in
    it, or is agreed on at once; and they agree before `ok` is the wait for an item."""
    text = _feeding()
    waits = re.findall(r"\bok = ([^;]*bar_wait[^;]*);(.{0,40})", text)
    assert len(waits) == 2
    for value, after in waits:
        assert value.startswith("ok && ") or after.startswith(" ok = __all_sync(~0u, ok);"), value
    assert re.search(r"ok = __all_sync\(~0u, ok\); if \(!ok\) break; \} ending = !read_item\(it\);", text)
    for value in re.findall(r"\bok = ([^;]*);", text):
        assert "bar_wait" in value or re.search(r"\bok\b", value), value


def test_nothing_goes_to_a_place_that_was_not_free():
    """A unit's place in the ring is written by a lane whose waits have all been good, and handed over likewise."""
    text = _feeding()
    ring = text[text.index("auto go = [&](auto octs_c"):text.index("using std::integral_constant")]
    assert ring.count("copy16(") == 1 and ring.count("if (ok) copy16(") == 1
    assert text.count("mbar_arrive(full + st)") == text.count("if (lane == 0 && (kI8 || ok)) mbar_arrive(full + st)") == 1
    assert "else if (!v && !second && ok && bads[at16])" in text
