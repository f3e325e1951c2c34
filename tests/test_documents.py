"""The documents' tables are whole: every run of table lines starts with a header and its rule. Needs no GPU."""
import os
import re

import pytest

from tests.conftest import ROOT


@pytest.mark.parametrize("name", ["README.md", "DESIGN.md"])
def test_tables_have_headers(name):
    lines = open(os.path.join(ROOT, name)).read().splitlines()
    fenced = False
    for i, line in enumerate(lines):
        fenced ^= line.startswith("```")
        if not fenced and line.startswith("|") and not (i and lines[i - 1].startswith("|")):
            assert i + 1 < len(lines) and re.fullmatch(r"\|[-:| ]+\|", lines[i + 1]), f"{name}:{i + 1}: {line[:80]}"
