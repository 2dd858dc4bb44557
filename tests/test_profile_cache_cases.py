"""The module that the committed ncu commands of the norm, cache and decode
kernels run: its case table and command-line checks, without a GPU, and every case
once on one."""
import pytest

from causal_linear_attention_chunked_b200 import profile_cache_cases


def test_cases_are_described():
    for name in profile_cache_cases.CASES:
        assert "\n  %s " % name in profile_cache_cases.__doc__


@pytest.mark.parametrize("argv", [[], ["nope"], ["norm", "read"]])
def test_bad_arguments_exit_with_usage(argv):
    with pytest.raises(SystemExit) as e:
        profile_cache_cases.main(argv)
    assert "usage" in str(e.value)


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(profile_cache_cases.CASES))
def test_case_runs(name, capsys):
    profile_cache_cases.main([name])
    assert capsys.readouterr().out == "ok\n"
