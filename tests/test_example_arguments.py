"""Arguments of the example decoder's command that do not go together are refused (CPU)."""
import sys

import pytest

from examples import block_decoder


def test_prefix_with_hybrid_is_refused(monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["block_decoder.py", "--hybrid", "--prefix", "100"])
    monkeypatch.setattr(block_decoder, "hybrid", lambda *a, **k: pytest.fail("the prefix was dropped"))
    with pytest.raises(SystemExit) as e:
        block_decoder.main()
    assert e.value.code == 2 and "--prefix" in capsys.readouterr().err


@pytest.mark.parametrize("argv,made", [([], ("small", 2, 100, 2, False)), (["--prefix", "0"], ("small", 2, 0, 2, False)),
                                       (["--hybrid", "--blocks", "3"], ("hybrid", 2, 3, False))])
def test_other_arguments_reach_the_decoder(monkeypatch, argv, made):
    class Made(Exception):
        pass

    def make(name):
        def f(*a):
            raise Made((name, *a))
        return f

    monkeypatch.setattr(sys, "argv", ["block_decoder.py", *argv])
    for name in ("small", "hybrid"):
        monkeypatch.setattr(block_decoder, name, make(name))
    with pytest.raises(Made) as e:
        block_decoder.main()
    assert e.value.args[0] == made
