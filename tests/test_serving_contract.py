"""What include/zha.h says of inputs that the attention kernels take differently: one path merges a walk's chunk ids in
a bitmap, others go through its list, so the header may ask for distinct ids and promise nothing of repeated ones."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def comment_of(name):
    with open(os.path.join(ROOT, "include", "zha.h")) as f:
        text = f.read()
    at = re.search(rf"^int {name}\(", text, re.M).start()
    return " ".join(text[text.rindex("/*", 0, at):at].replace(" * ", " ").split())


def test_attention_asks_for_distinct_ids():
    text = comment_of("zha_attend")
    assert "must be distinct" in text
    for name in ("zha_attend", "zha_attend_draft", "zha_attend_noalloc"):
        assert "counts once" not in comment_of(name)
    assert "as in zha_attend" in comment_of("zha_attend_draft")
