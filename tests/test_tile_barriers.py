"""The tile kernel's barriers, read from the source: taking down a barrier that was never set up is undefined."""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_verify_04_gb300",
                   "csrc", "attend_tile.cu")


def test_the_barriers_taken_down_are_those_set_up():
    with open(SRC) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    # one list, `each_bar`, names the barriers; setting up and taking down each go through it and nothing else does
    assert len(re.findall(r"\bmbar_init\(", text)) == 1 and len(re.findall(r"mbarrier\.inval", text)) == 1
    for what in (r"mbar_init\(b, arrivals\)", r"mbarrier\.inval"):
        assert re.search(r"each_bar\(\[\]\(uint64_t\* b, int[^{]*\{[^}]*" + what, text), what
    # and it names every barrier of the struct
    struct = text[text.index("struct TileBars {"):]
    struct = struct[:struct.index("};")]
    bars = re.findall(r"(\w+)(?:\[\d+\])?(?=[,;])", " ".join(re.findall(r"uint64_t[^;]*;", struct)))
    body = text[text.index("auto each_bar"):]
    body = body[:body.index("\n    };")]
    assert bars and all(re.search(r"f\(&B\." + b + r"\b", body) for b in bars), bars
