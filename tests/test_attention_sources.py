"""CPU checks of the attention kernels' sources: what can only be seen by reading."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_quantized_linear_gb300", "csrc")


def test_flags_between_blocks_are_only_touched_by_ordered_operations():
    # blocks set and read each other's flags at the same time: a plain store beside a load, volatile or not, is a data race
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "attn_kv_i4.cu")).read())
    assert re.search(r"st\.(relaxed|release)\.gpu", text) and re.search(r"ld\.(relaxed|acquire)\.gpu", text)
    assert "volatile unsigned long long" not in text
    assert not re.search(r"a\.flag\s*\[", text)
    uses = re.findall(r"(\w+)\(a\.flag\b", text)
    assert uses and set(uses) == {"set_flag", "flag_set"}
    assert len(re.findall(r"\ba\.flag\b", text)) == len(uses) + 1  # and where the host sets the pointer
    # set after a fence, with one behind it; looked at after a fence, with one before the parts are read
    assert re.search(r"__threadfence\(\);[^{}]*set_flag\(a\.flag[^{}]*kThere\);\s*__threadfence\(\);", text)
    assert re.search(r"__threadfence\(\);[^{}]*flag_set\(a\.flag[^{}]*__syncthreads_and\(there\)\) continue;\s*__threadfence\(\);", text)
