"""The README's tables are in one piece: a row of pipes that does not follow another row, or a header's rule, is
rendered as text.  CPU only."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tables_are_in_one_piece():
    lines = open(os.path.join(ROOT, "README.md")).read().splitlines()
    row = [ln.startswith("|") for ln in lines]
    for i, ln in enumerate(lines):
        if row[i] and (i == 0 or not row[i - 1]):   # a table's first line: its second is the rule
            assert i + 1 < len(lines) and re.fullmatch(r"\|(\s*:?-+:?\s*\|)+", lines[i + 1].strip()), f"line {i + 1}: {ln[:60]}"


def test_readme_names_every_entry_point_of_the_header():
    header = open(os.path.join(ROOT, "include", "jscan.h")).read()
    readme = open(os.path.join(ROOT, "README.md")).read()
    gated = [n for n in re.findall(r"^\s*(?:jscan_status|int64_t)\s+(jscan_\w+)\s*\(", header, re.M) if "gated" in n or "i8" in n or "quantize" in n]
    assert gated and [n for n in gated if n not in readme and not n.endswith(("_workspace", "_states"))] == []
