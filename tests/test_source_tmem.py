"""Loads from TMEM are asynchronous: their registers hold nothing before tcgen05.wait::ld. The compiler
takes them for written at the load, so each wait has to name the registers of the loads before it, or a
use may be moved above it. Checked on the text of csrc/ (no GPU)."""
import pathlib
import re

CSRC = pathlib.Path(__file__).resolve().parents[1] / "mixture_experts_layer_29_b200" / "csrc"
FILES = sorted(CSRC.glob("*.cu")) + sorted(CSRC.glob("*.cuh"))


def test_the_wait_stands_in_one_place():
    found = [(f.name, f.read_text().count("tcgen05.wait::ld.sync")) for f in FILES]
    assert [(n, c) for n, c in found if c] == [("common.cuh", 1)]
    text = (CSRC / "common.cuh").read_text()
    body = text[text.index("void tmem_ld_wait_for("):]
    assert '"+r"(r[i])' in body[:body.index("\n}\n")]


def test_each_wait_names_what_was_loaded():
    calls = 0
    for f in FILES:
        if f.name == "common.cuh":
            continue
        pending = []
        for m in re.finditer(r"tmem_ld_32x32b_x\d+\([^;]*, (\w+(?:\[\d\])?)\);|tmem_ld_wait\w*\(([^)]*)\)", f.read_text()):
            if m.group(1):
                pending.append(m.group(1))
            else:
                assert [a.strip() for a in m.group(2).split(",")] == pending and pending, (f.name, m.group(0), pending)
                pending, calls = [], calls + 1
        assert not pending, f.name
    assert calls >= 10
