"""The example that times an operator at a size of one's own."""

import importlib.util
import os
import re

import pytest

gpu = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "time_operators", os.path.join(ROOT, "examples", "time_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_cases_of_the_command_line():
    m = _example()
    c = m.case("lora", "128 4096 2048 16 64 requests fp16".split())
    assert (c["op"], c["M"], c["K"], c["N"], c["R"], c["L"]) == ("lora", 128, 4096, 2048, 16, 64)
    assert c["tokens"] == "requests" and c["dtype"] == "fp16"
    c = m.case("unsort", "1001 64 8 2 backward".split())
    assert (c["op"], c["M"], c["H"], c["E"], c["top_k"]) == ("unsort", 1001, 64, 8, 2)
    assert c["direction"] == "backward" and c["dtype"] == "bf16"
    assert m.case("gate", ["5", "8", "2"])["direction"] == "forward"
    with pytest.raises(SystemExit):
        m.case("gate", ["5", "8", "2", "sideways"])


@gpu
@pytest.mark.parametrize("args", ["lora 20 64 64 8 3", "gate 5 8 2 backward bf16",
                                  "sort 5 64 8 2 fp32", "unsort 5 63 8 2 backward fp16"])
def test_times_a_call(args, capsys):
    m = _example()
    try:
        m.main(args.split())
    finally:
        m.cases.own = False
    line = capsys.readouterr().out
    assert re.match(re.escape(args) + r": [\d.]+ us a call, floor [\d.]+ us\n$", line), line
