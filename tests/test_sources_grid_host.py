"""Persistent grids take the number of SMs from the device that they run on."""
import os
import re

from test_sources_host import CSRC


def test_the_slot_append_asks_the_device_for_its_sms():
    code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "kv_append.cu")).read())
    assert not re.search(r"\b152\b", code) and "num_sms" in code
