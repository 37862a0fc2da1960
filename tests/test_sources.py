"""CPU checks of the kernels' sources: what the compiler cannot see in inline assembly."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "expert_slot_cache_amd", "csrc")


def _statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*")) + glob.glob(os.path.join(CSRC, "*.cpp"))):
        for m in re.finditer(r"\basm\b\s*(?:volatile)?\s*\((.*?)\);", open(path).read(), flags=re.S):
            yield os.path.basename(path), m[1]


def test_inline_assembly_leaves_m0_to_the_compiler():
    """The compiler keeps no note of an M0 that a statement sets: it has to be an operand."""
    seen = 0
    for name, text in _statements():
        code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', text.split("::")[0]))
        assert not re.search(r"\bm0\b", code), (name, text)
        if "lds_dword" in code:                       # its LDS address is in M0
            assert "{m0}" in text, (name, text)
            seen += 1
    assert seen
