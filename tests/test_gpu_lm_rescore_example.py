"""The second pass's example, as a user without the repository's other folders runs it."""
import json
import sys

import pytest

from ctc_prefix_beam_amd import rescore

pytestmark = pytest.mark.gpu


def test_the_example_needs_the_package_alone(monkeypatch, capsys):
    for name in ("synth", "oracle", "tests"):
        monkeypatch.setitem(sys.modules, name, None)   # importing it raises
    path = list(sys.path)
    rescore.main()
    assert sys.path == path
    lines = capsys.readouterr().out.splitlines()
    assert [l.split(":")[0] for l in lines] == ["order before training", "loss per token",
                                                "order after training",
                                                "best of the first utterance"]
    loss = [float(v) for v in lines[1].split(":")[1].split()]
    assert len(loss) == 10 and loss[-1] < loss[0]
    assert sorted(json.loads(lines[0].split(":")[1])) == list(range(8))
