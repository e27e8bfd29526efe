"""The 4-bit attention's query is on its way to shared memory from an item's start: the CTA waits for it at the item's end whatever
happened in between (no entries, a wait that was given up), so that no copy outlives the CTA's use of its memory."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_lightning_gb300", "csrc")


def test_the_query_is_waited_for_on_every_way_to_an_items_end():
    with open(os.path.join(CSRC, "attn4_tc.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    loads = re.findall(r"tma_load_2d\([^;]*?\b(\w+), j \* 64", text)
    assert loads == ["q_staged"]                       # the only copies by TMA, in begin()
    begin, finish = text.index("auto begin = "), text.index("auto finish = ")
    head = text[finish:text.index("bool stopped", finish)]
    assert begin < text.index("tma_load_2d(") < finish
    drain = re.search(r"if \(([^;{]*)\) mbar_wait_drain\(q_staged, turn\);", head)
    assert drain and drain.group(1) == "warp == kMmaWarp"
    # every role leaves its items' loop behind finish() alone
    roles = text[text.index("if (warp >= kMmaWarp) {"):]
    assert roles.count("begin(item, it);") == roles.count("if (!finish(it)) break;") == 3
