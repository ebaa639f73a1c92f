"""profile_case.py's command line."""
import pytest

import profile_case


@pytest.fixture
def calls(monkeypatch):
    made = []
    for name in ("run", "run_operator"):
        monkeypatch.setattr(profile_case, name, lambda *a, _n=name, **kw: made.append((_n, a, kw)))
    return made


@pytest.mark.parametrize("line,call", [
    ("kvarn_131k", ("run", ("kvarn_131k",), {})),
    ("kvarn_131k num_seqs=1 ctx_lo=32768", ("run", ("kvarn_131k",), {"num_seqs": 1, "ctx_lo": 32768})),
    ("operators prefill_long", ("run_operator", ("operators", "prefill_long"), {})),
    ("more_operators prompt_long repeats=2", ("run_operator", ("more_operators", "prompt_long"), {"repeats": 2}))])
def test_arguments_are_numbers_by_name(calls, line, call):
    profile_case.main(line.split())
    assert calls == [call]


@pytest.mark.parametrize("line", ["operators prefill_long 2", "kvarn_131k 2", "more_operators prompt_long repeats=x"])
def test_other_words_are_refused(calls, line):
    with pytest.raises(ValueError):
        profile_case.main(line.split())
    assert calls == []
