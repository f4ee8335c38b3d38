"""Stores written in inline assembly keep the distance to what follows that the compiler keeps for its own: two wait
states between a store of more than 8 bytes and a write of its data registers, inside the same asm block."""

import glob
import os
import re

from bit_quantized_finetuning_amd import build as _build

WIDE = re.compile(r"(?:buffer|global|flat)_store_dwordx[34]\b[^;]*")


def _asm_strings(text):
    """The concatenated string literals of every asm statement."""
    for m in re.finditer(r"asm\s+volatile\s*\(((?:\s*\"(?:[^\"\\]|\\.)*\")+)", text):
        yield "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", m.group(1))).replace("\\n", "\n").replace("\\t", " ")


def test_wide_stores_are_followed_by_two_wait_states():
    seen = 0
    for path in sorted(glob.glob(os.path.join(_build.CSRC, "*"))):
        with open(path) as f:
            for asm in _asm_strings(f.read()):
                lines = [line.strip() for line in asm.splitlines()]
                for i, line in enumerate(lines):
                    if not WIDE.match(line):
                        continue
                    seen += 1
                    nop = re.fullmatch(r"s_nop (\d+)", lines[i + 1]) if i + 1 < len(lines) else None
                    assert nop and int(nop.group(1)) >= 1, f"{os.path.basename(path)}: {line}"
    assert seen >= 1
