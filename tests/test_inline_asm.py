"""Inline assembly of the HIP sources: what a statement overwrites is named in
its clobber list, and what the hardware wants between instructions that the
compiler does not see into is kept by the assembly (CPU only)."""
import glob
import os
import re
import subprocess

import pytest

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


def _scalars(text):
    out = set()
    for lo, hi, one in re.findall(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        out |= {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return out


def _too_close(lines):
    """Loads into LDS whose scalar address a vector instruction wrote fewer than
    5 wait states before, and all loads into LDS."""
    past, close, loads = [], [], 0  # (scalars a vector instruction wrote, wait states)
    for line in lines:
        code = line.split(";")[0].strip()
        if not code or code.startswith(".") or code.endswith(":"):
            continue
        op, _, args = code.partition(" ")
        if op.startswith("global_load_lds"):
            loads += 1
            states = 0
            for wrote, n in reversed(past):
                if states >= 5:
                    break
                if wrote & _scalars(args):
                    close.append(code)
                states += n
        first = args.split(",")[0]
        past.append((_scalars(first) if op.startswith("v_") else set(), int(args) + 1 if op == "s_nop" else 1))
        del past[:-8]
    return close, loads


def test_scan_finds_an_address_that_is_too_young():
    young = ["v_readfirstlane_b32 s4, v1", "s_mov_b32 m0, s9", "s_nop 0", "global_load_lds_dwordx4 v2, s[4:5]"]
    assert _too_close(young) == ([young[-1]], 1)
    assert _too_close([young[0], "s_nop 4", *young[1:]]) == ([], 1)
    assert _too_close([young[0].replace("s4", "s7"), *young[1:]]) == ([], 1)


def test_scalar_addresses_of_loads_into_lds_are_old_enough(tmp_path):
    from combine_ep_layout_03_amd import build as b

    try:
        hipcc = b.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    out = tmp_path / "linear.s"
    flags = [f for f in b.HIPCC_FLAGS if f != "-shared"]
    res = subprocess.run([hipcc, *flags, "-I", b.INCLUDE, "-I", b.CSRC, "-S", "--cuda-device-only",
                          os.path.join(b.CSRC, "ep_linear.hip"), "-o", str(out)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    close, loads = _too_close(out.read_text().splitlines())
    assert loads > 100 and close == []
