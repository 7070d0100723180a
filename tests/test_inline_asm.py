"""Inline assembly of the HIP sources: what a statement overwrites is named in
its clobber list (CPU only)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _statements():
    for path in sorted(glob.glob(os.path.join(ROOT, "combine_ep_layout_03_amd", "csrc", "*"))):
        src = open(path).read()
        for m in re.finditer(r"\basm\s+volatile\s*\(", src):
            depth, i, quoted = 1, m.end(), False
            while depth:
                c = src[i]
                if c == '"' and src[i - 1] != "\\":
                    quoted = not quoted
                elif not quoted:
                    depth += (c == "(") - (c == ")")
                i += 1
            yield os.path.basename(path), src[m.end():i - 1]


def test_statements_that_write_m0_name_it():
    seen = 0
    for name, text in _statements():
        code, *rest = re.split(r'"\s*:', text, maxsplit=1)
        if re.search(r"\b(s_mov_b32|s_add_u32|s_lshl_b32)\s+m0\b", code):
            seen += 1
            assert '"m0"' in text[len(code):], f"{name}: {text}"
    assert seen >= 2  # the loads into LDS
