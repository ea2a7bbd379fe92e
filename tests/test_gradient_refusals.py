"""What is not of the kind that an operator takes is refused as such, before anything is enqueued.
Nothing here reaches a GPU."""
import pytest
import torch

from test_gradient_host import NAMES, h, operands, stored
from test_training_host import calls, placed  # noqa: F401 (a fixture)

# what no operand may be, whatever it is called
NEVER = {"a list": [1.0], "a text": "x", "on the host": torch.zeros(4, 24),
         "64 bits": placed(4, 24, dtype=torch.float64)}
# what some operands are, and others are not
TENSOR, CHECKPOINT = h(4, 24), stored(4, 24)


@pytest.mark.parametrize("name", NAMES)
def test_operands_of_another_kind_are_refused(name, calls):  # noqa: F811
    for which, right in operands(name)[1].items():
        kinds = dict(NEVER)
        if which == "ws":
            del kinds["64 bits"]  # bytes of any type
        if which != "x" or name == "restore8":
            kinds["the other kind"] = TENSOR if hasattr(right, "codes") else CHECKPOINT
        for kind, wrong in kinds.items():
            f, args, _ = operands(name)
            args[which] = wrong
            with pytest.raises((TypeError, ValueError)):
                f(**args)
                print(which, kind)
    assert calls == []


def test_what_stands_for_an_activation_is_asked_for_by_name(calls):  # noqa: F811
    for name, which in (("restore8", "x"), ("checkpoint8", "out")):
        f, args, _ = operands(name)
        args[which] = TENSOR
        with pytest.raises(TypeError, match=f"{which} must be a Checkpoint8"):
            f(**args)
    assert calls == []
