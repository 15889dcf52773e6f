"""That the layer's checks accept the definition and reject wrong absorbed attention."""
import pytest

from latent_layer import Definition, Layer

FAULTS = ["no rotary part", "16 keys lost", "no causal mask", "uniform weights"]


def test_the_definition_passes():
    s = Layer("cpu")
    s.run(Definition())
    s.check_rows()
    s.check_absorbed()
    s.check_expanded()
    s.check_formula()


@pytest.mark.parametrize("fault", FAULTS)
def test_a_wrong_absorbed_form_is_rejected(fault):
    s = Layer("cpu")
    s.run(Definition(fault))
    with pytest.raises(AssertionError):
        s.check_absorbed()
    with pytest.raises(AssertionError):
        s.check_formula()


def test_rows_that_were_not_turned_are_rejected():
    s = Layer("cpu")
    s.run(Definition("rows not turned"))
    with pytest.raises(AssertionError):
        s.check_rows()
