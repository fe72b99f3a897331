"""Every bit that a kernel sets in the device error word is named where the header describes
q8_device_error."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_header_names_every_bit_of_the_error_word():
    with open(os.path.join(ROOT, "include", "q8.h")) as f:
        said = re.search(r"q8_device_error -- .*?\*/", f.read(), re.S)[0]
    bits = set()
    for path in glob.glob(os.path.join(ROOT, "q8_int8_block_gb300", "csrc", "*")):
        with open(path) as f:
            bits |= {int(n) for n in re.findall(r"\bkErr\w+ = 1u << (\d+)", f.read())}
    assert {0, 1} <= bits
    assert {int(n) for n in re.findall(r"\bbit (\d+)", said)} == bits
