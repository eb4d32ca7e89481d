"""A register that tcgen05.ld fills holds its value only behind tcgen05.wait::ld: the wait
has to name the registers, or the compiler may use them before it."""
import glob
import os
import re

import post_weight_quantization_11_b200 as pkg


def test_every_wait_for_a_tmem_load_names_its_registers():
    found = 0
    for path in glob.glob(os.path.join(os.path.dirname(pkg.__file__), "csrc", "*.cu*")):
        src = open(path, encoding="utf-8").read()
        for load in re.finditer(r'asm volatile\(\s*"tcgen05\.ld\..*?\);\n', src, re.S):
            regs = re.findall(r'"=r"\((\w+\[\d+\])\)', load.group())
            wait = re.search(r'asm volatile\("tcgen05\.wait::ld\..*?\);\n', src[load.end():], re.S).group()
            assert regs and re.findall(r'"\+r"\((\w+\[\d+\])\)', wait) == regs, (path, load.group())
            found += 1
        assert len(re.findall(r'"tcgen05\.wait::ld', src)) == len(re.findall(r'"tcgen05\.ld\.', src)), path
    assert found >= 2
