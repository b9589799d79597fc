"""No variable of a CUDA source has the name of the parameter of a template that it stands in: C++ does not allow it (a
compiler that lets it pass takes the variable from there on).  No GPU is needed: the sources are read."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).parents[1] / "deepseek_v4_compressed_wkv_gb300" / "csrc"


def bodies(text):
    """(parameter names, body) of every template with a body."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\btemplate\s*<([^<>]*)>", text):
        names = [re.sub(r"=.*", "", p).split()[-1].lstrip(".") for p in m[1].split(",") if p.strip()]
        begin = min((i for i in (text.find("{", m.end()), ) if i >= 0), default=-1)
        if begin < 0 or 0 <= text.find(";", m.end()) < begin:
            continue
        depth = 0
        for end in range(begin, len(text)):
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            if depth == 0:
                break
        yield names, text[begin:end]


@pytest.mark.parametrize("path", sorted(CSRC.glob("*.cu*")), ids=lambda p: p.name)
def test_template_parameters_keep_their_names(path):
    for names, body in bodies(path.read_text()):
        for name in names:
            again = re.search(r"\b(int|bool|auto|float|uint32_t|uint64_t|uint8_t|long)\s+" + re.escape(name) + r"\s*[=;,]", body)
            assert not again, again[0]
