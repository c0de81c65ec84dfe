"""Bounded waits of the tensor-memory attention, read from its source: a warp
whose lanes go on to shuffles, ballots or barriers of the whole warp leaves a
wait as a whole. (A lane that gave up on its own would leave its neighbours in
them for good, so this is read and not run.)"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_verification_83_gb300", "csrc")


def source():
    with open(os.path.join(CSRC, "dflash_attention_tc.cu")) as f:
        return re.sub(r"//.*", "", f.read())


def test_load_warps_give_up_together():
    s = source()
    waits = re.findall(r"(\w+)\(&S\.empty\[st\], ", s)
    assert len(waits) == 2 and set(waits) == {"warp_wait"}
    body = re.search(r"bool warp_wait\([^)]*\)\s*\{(.*?)\n\}", s, re.S).group(1)
    assert re.search(r"return __all_sync\(0xffffffffu, tc_wait\(", body)


def test_softmax_warps_give_up_together():
    """Every wait of the softmax's part is followed by a vote, or is one."""
    s = source()
    part = s[s.index("uint32_t syncs = 0;"):s.index("if (!ok && lane == 0) raise_status")]
    for m in re.finditer(r"product_done\(j|tc_wait\(&S\.(s_full|full)", part):
        after = part[m.start():m.start() + 220]
        assert "__all_sync(0xffffffffu, ok)" in after, after
    body = re.search(r"bool softmax_sync\([^)]*\)\s*\{(.*?)\n\}", s, re.S).group(1)
    assert "__all_sync" in body
