"""moe_status_string: each status by its name; the bounds error names both ranges of ids."""
from routing_dispatch_grouped_gb300 import moe


def test_status_strings():
    text = {k: moe.lib().moe_status_string(k).decode() for k in moe.STATUS}
    assert all(text[k].startswith(name) for k, name in moe.STATUS.items())
    assert "expert id outside [0, E)" in text[5] and "token id outside [0, V)" in text[5]
    assert moe.lib().moe_status_string(99).decode().startswith("unknown")
