"""Names and constants that the header and the binding share; the texts of the statuses."""
import os
import re

from routing_dispatch_grouped_gb300 import moe


def test_status_strings():
    text = {k: moe.lib().moe_status_string(k).decode() for k in moe.STATUS}
    assert all(text[k].startswith(name) for k, name in moe.STATUS.items())
    assert "expert id outside [0, E)" in text[5] and "token id outside [0, V)" in text[5]
    assert moe.lib().moe_status_string(99).decode().startswith("unknown")


def test_constants_of_the_binding_are_the_headers():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "moe.h")) as f:
        text = f.read()
    assert int(re.search(r"#define MOE_ADAMW_BLOCK (\d+)", text).group(1)) == moe.ADAMW_BLOCK
    for name in ("NORM_RMS", "IDS_64", "WGRAD_BF16"):
        assert int(re.search(rf"MOE_{name} = (\d+)u", text).group(1)) == getattr(moe, name)
